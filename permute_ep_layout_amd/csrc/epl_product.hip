// libepl.so host side of the experts' products: argument checks and launches
// of epl_expert_product and epl_expert_weight_grad (include/epl.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epl.h"
#include "epl_product_kernels.h"

namespace {

namespace P = epl_product;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launch_status() { return hipGetLastError() == hipSuccess ? EPL_OK : EPL_EHIP; }

// Offsets within one expert's weight and within a tile are 32-bit.
constexpr int32_t kMaxCols = 1 << 20;
constexpr int64_t kMaxWeight = int64_t(1) << 29;

bool is_grad(int act)
{
    return act == EPL_ACT_SILU_GRAD || act == EPL_ACT_GELU_GRAD || act == EPL_ACT_SWIGLU_GRAD;
}

bool desc_ok(const epl_product_desc *p)
{
    if (!p || p->reserved != 0)
        return false;
    if (p->num_experts < 1 || p->num_experts > P::kMaxExperts)
        return false;
    if (p->num_rows < 0 || p->num_rows > INT32_MAX || p->expected_rows < 0)
        return false;
    if (p->in_cols < 8 || p->in_cols % 8 != 0 || p->in_cols > kMaxCols || p->out_cols < 8 ||
        p->out_cols % 8 != 0 || p->out_cols > kMaxCols)
        return false;
    if ((int64_t)p->in_cols * p->out_cols > kMaxWeight)
        return false;
    if (p->activation < EPL_ACT_NONE || p->activation > EPL_ACT_SWIGLU_GRAD)
        return false;
    if (p->activation == EPL_ACT_SWIGLU && p->out_cols % 16 != 0)
        return false;
    if (p->out_type != EPL_OUT_F32 && p->out_type != EPL_OUT_BF16)
        return false;
    return p->weight_layout == EPL_WEIGHT_OUT_IN || p->weight_layout == EPL_WEIGHT_IN_OUT;
}

int num_cus()
{
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) {
        (void)hipGetLastError();
        return 256;
    }
    return n;
}

template <int BM, int BN, P::Form FORM>
int launch_tiles(const P::Args &a, int64_t tiles, hipStream_t s)
{
    // one workgroup a CU, striding over the tiles
    const int64_t grid = std::min<int64_t>(tiles, num_cus());
    hipLaunchKernelGGL((P::tile_kernel<BM, BN, FORM>), dim3((unsigned)grid), dim3(P::kTileThreads), 0,
                       s, a);
    return launch_status();
}

}  // namespace

extern "C" {

int epl_product_validate(const epl_product_desc *p) { return desc_ok(p) ? EPL_OK : EPL_EINVAL; }

int epl_expert_product(const epl_product_desc *p, const uint16_t *x, const uint16_t *weight,
                       const float *bias, const uint16_t *residual,
                       const int32_t *expert_start_loc, const int32_t *num_tokens_per_expert,
                       uint16_t *pre, void *y, void *stream)
{
    if (!desc_ok(p))
        return EPL_EINVAL;
    const bool grad = is_grad(p->activation);
    if (grad && (bias || residual))
        return EPL_EINVAL;
    if (!weight || !aligned(weight, 16) || !expert_start_loc || !aligned(expert_start_loc, 4) ||
        !num_tokens_per_expert || !aligned(num_tokens_per_expert, 4) || !aligned(bias, 16) ||
        !aligned(residual, 16) || !aligned(pre, 16))
        return EPL_EINVAL;
    if (p->num_rows == 0)
        return EPL_OK;
    if (!x || !aligned(x, 16) || !y || !aligned(y, 16) || (grad && !pre))
        return EPL_EINVAL;
    P::Args a{};
    a.p = reinterpret_cast<const __bf16 *>(x);
    a.q = reinterpret_cast<const __bf16 *>(weight);
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

    // The counts are on the GPU: the kernel is chosen by the rows that the
    // caller expects an expert to have on average.
    const int64_t rows = p->expected_rows > 0 ? std::min(p->expected_rows, p->num_rows) : p->num_rows;
    const int64_t avg = (rows + a.E - 1) / a.E;
    const bool swiglu = a.act == EPL_ACT_SWIGLU;
    if (p->weight_layout == EPL_WEIGHT_OUT_IN && avg <= 64) {
        const int nb = swiglu ? (a.N / 2 + 15) / 16 : (a.N + 31) / 32;
        hipLaunchKernelGGL(P::few_rows_kernel, dim3((unsigned)nb, (unsigned)a.E),
                           dim3(P::kFewThreads), 0, s, a);
        return launch_status();
    }
    // Tile rows: 256 reuse the weights most; 128 make more tiles. Rounds of
    // one tile a CU are compared, a tile of 128 rows at 0.65 of the time of
    // one of 256 (measured: 64 experts of 192 rows, 4096 -> 2048, 297 us in 2
    // rounds of 256 against 381 us in 4 of 128; 8 experts of 192 rows, 7168
    // -> 4096, 198 us against 166 us in one round each).
    const int64_t cus = num_cus(), ntn = (a.N + 255) / 256;
    auto rounds = [&](int64_t bm) { return ((avg + bm - 1) / bm * a.E * ntn + cus - 1) / cus; };
    const bool tall = rounds(256) * 100 <= rounds(128) * 65;
    auto tiles = [&](int bm) { return (p->num_rows / bm + a.E) * ntn; };
    if (p->weight_layout == EPL_WEIGHT_OUT_IN)
        return tall ? launch_tiles<256, 256, P::kForward>(a, tiles(256), s)
                    : launch_tiles<128, 256, P::kForward>(a, tiles(128), s);
    return tall ? launch_tiles<256, 256, P::kDataGrad>(a, tiles(256), s)
                : launch_tiles<128, 256, P::kDataGrad>(a, tiles(128), s);
}

int epl_expert_weight_grad(const epl_product_desc *p, const uint16_t *grad, const uint16_t *x,
                           const int32_t *expert_start_loc, const int32_t *num_tokens_per_expert,
                           int accumulate, void *grad_weight, float *grad_bias, void *stream)
{
    if (!desc_ok(p) || p->activation != EPL_ACT_NONE || p->weight_layout != EPL_WEIGHT_OUT_IN ||
        (accumulate != 0 && accumulate != 1))
        return EPL_EINVAL;
    if (!expert_start_loc || !aligned(expert_start_loc, 4) || !num_tokens_per_expert ||
        !aligned(num_tokens_per_expert, 4) || !grad_weight || !aligned(grad_weight, 16) ||
        !aligned(grad_bias, 4))
        return EPL_EINVAL;
    if (p->num_rows > 0 && (!x || !aligned(x, 16) || !grad || !aligned(grad, 16)))
        return EPL_EINVAL;
    P::Args a{};
    a.p = reinterpret_cast<const __bf16 *>(grad);
    a.q = reinterpret_cast<const __bf16 *>(x);
    a.y = grad_weight;
    a.start = expert_start_loc;
    a.count = num_tokens_per_expert;
    a.rows = p->num_rows;
    a.E = p->num_experts;
    a.K = p->in_cols;
    a.N = p->out_cols;
    a.act = EPL_ACT_NONE;
    a.out_f32 = p->out_type == EPL_OUT_F32;
    a.accumulate = accumulate;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t tiles = (int64_t)a.E * ((a.N + 255) / 256) * ((a.K + 255) / 256);
    int rc = launch_tiles<256, 256, P::kWeightGrad>(a, tiles, s);
    if (rc == EPL_OK && grad_bias) {
        hipLaunchKernelGGL(P::bias_grad_kernel, dim3((unsigned)((a.N + 63) / 64), (unsigned)a.E),
                           dim3(P::kBiasThreads), 0, s, a, grad_bias);
        rc = launch_status();
    }
    return rc;
}

}  // extern "C"
