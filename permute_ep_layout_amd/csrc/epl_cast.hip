// libepl.so host side of the 8-bit casts: argument checks and launches of
// epl_quantize, epl_dequantize and epl_quantize_weight (include/epl.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epl.h"
#include "epl_cast_kernels.h"

namespace {

namespace C = epl_cast;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launch_status() { return hipGetLastError() == hipSuccess ? EPL_OK : EPL_EHIP; }

constexpr int32_t kMaxCols = 1 << 20;
constexpr int64_t kMaxRows = INT32_MAX - 1023;   // rows are stepped through in 32 bits

bool type_ok(int t) { return t == EPL_OUT_F32 || t == EPL_OUT_BF16; }

bool cast_ok(const epl_cast_desc *p)
{
    if (!p || p->reserved != 0 || p->reserved2 != 0)
        return false;
    if (p->num_rows < 0 || p->num_rows > kMaxRows)
        return false;
    if (p->num_experts < 0 || p->num_experts > epl_product::kMaxExperts)
        return false;
    if (p->cols < 16 || p->cols % 16 != 0 || p->cols > kMaxCols || !type_ok(p->value_type))
        return false;
    if (p->activation != EPL_ACT_NONE && p->activation != EPL_ACT_SWIGLU)
        return false;
    if (p->scale_format == EPL_SCALE_F32_RECT)
        return p->rows_per_expert >= 1 && p->num_rows % p->rows_per_expert == 0;
    return p->rows_per_expert == 0 &&
           (p->scale_format == EPL_SCALE_F32 || p->scale_format == EPL_SCALE_UE8M0);
}

int64_t weight_blocks(const epl_weight_cast_desc &p)
{
    return (int64_t)p.num_experts * ((p.in_cols + 127) / 128) * ((p.out_cols + 127) / 128);
}

bool weight_ok(const epl_weight_cast_desc *p)
{
    if (!p || p->reserved != 0 || p->num_experts < 1 || p->num_experts > epl_product::kMaxExperts)
        return false;
    if (p->in_cols < 16 || p->in_cols % 16 != 0 || p->in_cols > kMaxCols || p->out_cols < 1 ||
        p->out_cols > kMaxCols || !type_ok(p->value_type))
        return false;
    return weight_blocks(*p) <= INT32_MAX &&
           (p->scale_format == EPL_SCALE_F32 || p->scale_format == EPL_SCALE_UE8M0);
}

C::Args args_of(const epl_cast_desc &p, uint8_t *codes, void *scale, const int32_t *start,
                const int32_t *count)
{
    C::Args a{};
    a.codes = codes;
    a.scales = C::Scales{scale, p.scale_format, (p.cols + C::kGroup - 1) / C::kGroup,
                         p.rows_per_expert, p.num_rows};
    a.start = p.num_experts ? start : nullptr;
    a.count = count;
    a.rows = p.num_rows;
    a.E = std::max(p.num_experts, 1);
    a.C = p.cols;
    return a;
}

// Blocks are both or neither; the rest that both directions check.
bool pointers_ok(const epl_cast_desc &p, const void *values, const void *codes, const void *scale,
                 const int32_t *start, const int32_t *count)
{
    if (p.num_experts > 0 && (!start || !count || !aligned(start, 4) || !aligned(count, 4)))
        return false;
    return values && aligned(values, 16) && codes && aligned(codes, 16) && scale && aligned(scale, 4);
}

unsigned grid_of(const C::Args &a)
{
    const int64_t tiles = (a.rows / C::kRows + a.E) * ((a.C + C::kCols - 1) / C::kCols);
    return (unsigned)std::min<int64_t>(tiles, C::kGrid);
}

}  // namespace

extern "C" {

int epl_cast_validate(const epl_cast_desc *p) { return cast_ok(p) ? EPL_OK : EPL_EINVAL; }

int epl_weight_cast_validate(const epl_weight_cast_desc *p)
{
    return weight_ok(p) ? EPL_OK : EPL_EINVAL;
}

int epl_quantize(const epl_cast_desc *p, const void *x, const int32_t *expert_start_loc,
                 const int32_t *num_tokens_per_expert, uint8_t *codes, void *scale, void *stream)
{
    if (!cast_ok(p))
        return EPL_EINVAL;
    if (p->num_rows == 0)
        return EPL_OK;
    if (!pointers_ok(*p, x, codes, scale, expert_start_loc, num_tokens_per_expert))
        return EPL_EINVAL;
    C::Args a = args_of(*p, codes, scale, expert_start_loc, num_tokens_per_expert);
    a.x = x;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(grid_of(a)), threads(C::kThreads);
    const bool gated = p->activation == EPL_ACT_SWIGLU, f32 = p->value_type == EPL_OUT_F32;
    if (gated && f32)
        hipLaunchKernelGGL((C::quantize_kernel<float, true>), grid, threads, 0, s, a);
    else if (gated)
        hipLaunchKernelGGL((C::quantize_kernel<__bf16, true>), grid, threads, 0, s, a);
    else if (f32)
        hipLaunchKernelGGL((C::quantize_kernel<float, false>), grid, threads, 0, s, a);
    else
        hipLaunchKernelGGL((C::quantize_kernel<__bf16, false>), grid, threads, 0, s, a);
    return launch_status();
}

int epl_dequantize(const epl_cast_desc *p, const uint8_t *codes, const void *scale,
                   const int32_t *expert_start_loc, const int32_t *num_tokens_per_expert, void *y,
                   void *stream)
{
    if (!cast_ok(p) || p->activation != EPL_ACT_NONE)
        return EPL_EINVAL;
    if (p->num_rows == 0)
        return EPL_OK;
    if (!pointers_ok(*p, y, codes, scale, expert_start_loc, num_tokens_per_expert))
        return EPL_EINVAL;
    C::Args a = args_of(*p, const_cast<uint8_t *>(codes), const_cast<void *>(scale),
                        expert_start_loc, num_tokens_per_expert);
    a.y = y;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(grid_of(a)), threads(C::kThreads);
    if (p->value_type == EPL_OUT_F32)
        hipLaunchKernelGGL((C::dequantize_kernel<float>), grid, threads, 0, s, a);
    else
        hipLaunchKernelGGL((C::dequantize_kernel<__bf16>), grid, threads, 0, s, a);
    return launch_status();
}

int epl_quantize_weight(const epl_weight_cast_desc *p, const void *weight, uint8_t *codes,
                        void *scale, void *stream)
{
    if (!weight_ok(p))
        return EPL_EINVAL;
    const bool power = p->scale_format == EPL_SCALE_UE8M0;
    if (!weight || !aligned(weight, 16) || !codes || !aligned(codes, 16) || !scale ||
        !aligned(scale, power ? 1 : 4))
        return EPL_EINVAL;
    const C::WeightArgs a{weight, codes, scale, p->out_cols, p->in_cols, power, weight_blocks(*p)};
    const dim3 grid((unsigned)std::min<int64_t>(a.blocks, C::kWeightGrid)), threads(C::kThreads);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p->value_type == EPL_OUT_F32)
        hipLaunchKernelGGL((C::quantize_weight_kernel<float>), grid, threads, 0, s, a);
    else
        hipLaunchKernelGGL((C::quantize_weight_kernel<__bf16>), grid, threads, 0, s, a);
    return launch_status();
}

}  // extern "C"
