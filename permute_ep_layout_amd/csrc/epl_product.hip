// libepl.so host side of the experts' products: argument checks and launches
// of epl_expert_product and epl_expert_weight_grad (include/epl.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epl.h"
#include "epl_product_host.h"
#include "epl_product_kernels.h"

namespace epl_product {

// --------------------------------------------------------- bias gradient --
//
// db[e, n] = sum over the expert's rows of d[p, n], in binary32. A workgroup
// takes 64 columns (8 lanes of 8) of one expert; its 32 row lanes add rows
// 32 apart and are added in order through LDS. 12288 rows over 64 experts, 2048
// columns: 10 us. Rows are not shared over workgroups, so that one expert of
// 16384 rows and 64 columns takes 142 us, four times its weight gradient.

constexpr int kBiasThreads = 256;

__global__ __launch_bounds__(kBiasThreads) void bias_grad_kernel(Args a, float *db)
{
    __shared__ float red[32][65];
    const int e = blockIdx.y, tid = threadIdx.x, c = tid & 7, y = tid >> 3;
    const int n = blockIdx.x * 64 + c * 8;
    int64_t lo;
    const int cnt = block_of(a, e, lo);
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n < a.N) {
        for (int m = y; m < cnt; m += 32) {
            float v[8];
            load_bf16<8>(a.p + (lo + m) * a.N + n, v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] += v[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        red[y][c * 8 + i] = s[i];
    __syncthreads();
    if (tid < 64 && (int)blockIdx.x * 64 + tid < a.N) {
        float t = 0;
        for (int i = 0; i < 32; ++i)
            t += red[i][tid];
        float *out = db + (int64_t)e * a.N + blockIdx.x * 64 + tid;
        *out = a.accumulate ? *out + t : t;
    }
}

}  // namespace epl_product

namespace {

namespace P = epl_product;
namespace H = epl_product_host;

using namespace H;

// Rows an expert, on average, up to which the weights are read straight from
// memory.
constexpr int64_t kFewRows = 12;

constexpr int64_t kMaxWeight = int64_t(1) << 29;     // elements of an expert's

bool desc_ok(const epl_product_desc *p)
{
    if (!p || p->reserved != 0)
        return false;
    if (p->num_experts < 1 || p->num_experts > P::kMaxExperts)
        return false;
    if (p->num_rows < 0 || p->num_rows > kMaxRows || p->expected_rows < 0)
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

// The costs of the bf16 tiles: a round of large tiles takes 13 us and 1.55 a
// stage, one of as many small ones as the GPU holds (half their outputs) 7 and
// 1.1: large tiles read the operands half as often, small ones leave less idle
// where the last round is not full.
constexpr Cost cost_of(Kind k) { return k == kLarge ? Cost{13.0, 1.55} : Cost{7.0, 1.1}; }

int max_parts(int64_t depth) { return H::max_parts(depth, P::kTileK); }

int stages_of(int64_t depth) { return H::stages_of(depth, P::kTileK); }

double tiles_time(Kind k, int64_t m, int64_t n, int64_t experts, int64_t depth)
{
    return H::tiles_time(k, m, n, experts, depth, P::kTileK, cost_of(k));
}

// The faster kind by that. Measured (large, small), us: 8 experts of 4096
// rows, 7168 -> 4096: 1474, 1811; 64 of 192, 4096 -> 2048: 277, 320; 8 of 256,
// 7168 -> 4096 (128 large tiles): 149, 158; 8 of 768, 1024 -> 2048: 47, 58;
// but 64 of 128, 4096 -> 2048: 256, 218; 8 of 512, 2048 -> 2048 (128 large
// tiles): 58, 44; 16 of 500, 512 -> 640: 38, 21; weight gradients of 8
// experts, 1536 x 2048, of 256 rows: 40, 32, of 1024: 78, 63, but of 4096:
// 190, 194.
Kind tiles_for(int64_t m, int64_t n, int64_t experts, int64_t depth)
{
    return tiles_time(kLarge, m, n, experts, depth) <= tiles_time(kSmall, m, n, experts, depth) ? kLarge
                                                                                                : kSmall;
}

int64_t expected_rows(const epl_product_desc &p)
{
    return p.expected_rows > 0 ? std::min(p.expected_rows, p.num_rows) : p.num_rows;
}

int64_t average_rows(const epl_product_desc &p)
{
    return (expected_rows(p) + p.num_experts - 1) / p.num_experts;
}

Kind kind_of(const epl_product_desc &p)
{
    const int64_t avg = average_rows(p);
    if (p.weight_layout == EPL_WEIGHT_OUT_IN && avg <= kFewRows)
        return kFew;
    return tiles_for(avg, p.out_cols, p.num_experts, p.in_cols);
}

// The depth of a weight gradient's contraction is the expert's rows.
int64_t grad_depth(const epl_product_desc &p) { return expected_rows(p) / p.num_experts; }

Kind grad_kind_of(const epl_product_desc &p)
{
    return tiles_for(p.out_cols, p.in_cols, p.num_experts, grad_depth(p));
}

int64_t product_tiles(const epl_product_desc &p, Kind k)
{
    return H::product_tiles(p.num_rows, p.num_experts, p.out_cols, k);
}

int64_t grad_tiles(const epl_product_desc &p, Kind k)
{
    return (int64_t)p.num_experts * ((p.out_cols + side_of(k) - 1) / side_of(k)) *
           ((p.in_cols + side_of(k) - 1) / side_of(k));
}

template <int SIDE, P::Form FORM>
int launch_tiles(const P::Args &a, int64_t tiles, hipStream_t s)
{
    const bool split = a.ws && a.max_parts > 1;
    const int grid = tile_grid(a, tiles, SIDE, split);
    constexpr int threads = P::tile_threads(SIDE);
    hipLaunchKernelGGL((P::tile_kernel<SIDE, SIDE, FORM>), dim3((unsigned)grid), dim3(threads), 0, s, a);
    int rc = launch_status();
    if (rc == EPL_OK && split) {
        constexpr int pieces = SIDE / P::kWavesM / 16;
        hipLaunchKernelGGL((P::join_kernel<SIDE, SIDE, FORM>), dim3(pieces, join_grid(tiles, grid)),
                           dim3(threads), 0, s, a, grid);
        rc = launch_status();
    }
    return rc;
}

template <P::Form FORM>
int launch_kind(Kind k, const P::Args &a, int64_t tiles, hipStream_t s)
{
    return k == kSmall ? launch_tiles<128, FORM>(a, tiles, s) : launch_tiles<256, FORM>(a, tiles, s);
}

}  // namespace

extern "C" {

int epl_product_validate(const epl_product_desc *p) { return desc_ok(p) ? EPL_OK : EPL_EINVAL; }

size_t epl_product_workspace_bytes(const epl_product_desc *p)
{
    if (!desc_ok(p))
        return 0;
    const Kind k = kind_of(*p);
    return tile_workspace(k, product_tiles(*p, k), max_parts(p->in_cols));
}

size_t epl_weight_grad_workspace_bytes(const epl_product_desc *p)
{
    if (!desc_ok(p))
        return 0;
    const Kind k = grad_kind_of(*p);
    return tile_workspace(k, grad_tiles(*p, k), max_parts(grad_depth(*p)));
}

int epl_expert_product(const epl_product_desc *p, const uint16_t *x, const uint16_t *weight,
                       const float *bias, const uint16_t *residual,
                       const int32_t *expert_start_loc, const int32_t *num_tokens_per_expert,
                       uint16_t *pre, void *y, void *workspace, void *stream)
{
    if (!desc_ok(p))
        return EPL_EINVAL;
    const bool grad = is_grad(p->activation);
    if (grad && (bias || residual))
        return EPL_EINVAL;
    if (!weight || !aligned(weight, 16) || !expert_start_loc || !aligned(expert_start_loc, 4) ||
        !num_tokens_per_expert || !aligned(num_tokens_per_expert, 4) || !aligned(bias, 16) ||
        !aligned(residual, 16) || !aligned(pre, 16) || !aligned(workspace, 256))
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
    const Kind k = kind_of(*p);
    if (k == kFew) {
        // 16 waves a workgroup where 4 would leave the GPU mostly empty
        const int nb = (a.N + P::kFewCols - 1) / P::kFewCols;
        const dim3 grid((unsigned)nb, (unsigned)a.E);
        if ((int64_t)nb * a.E <= kCus)
            hipLaunchKernelGGL((P::few_rows_kernel<16>), grid, dim3(1024), 0, s, a);
        else
            hipLaunchKernelGGL((P::few_rows_kernel<4>), grid, dim3(256), 0, s, a);
        return launch_status();
    }
    a.max_parts = max_parts(a.K);
    a.stages = stages_of(a.K);
    use_workspace(a, a.max_parts > 1 ? workspace : nullptr);
    const int64_t tiles = product_tiles(*p, k);
    return p->weight_layout == EPL_WEIGHT_OUT_IN ? launch_kind<P::kForward>(k, a, tiles, s)
                                                 : launch_kind<P::kDataGrad>(k, a, tiles, s);
}

int epl_expert_weight_grad(const epl_product_desc *p, const uint16_t *grad, const uint16_t *x,
                           const int32_t *expert_start_loc, const int32_t *num_tokens_per_expert,
                           int accumulate, void *grad_weight, float *grad_bias, void *workspace,
                           void *stream)
{
    if (!desc_ok(p) || p->activation != EPL_ACT_NONE || p->weight_layout != EPL_WEIGHT_OUT_IN ||
        (accumulate != 0 && accumulate != 1))
        return EPL_EINVAL;
    if (!expert_start_loc || !aligned(expert_start_loc, 4) || !num_tokens_per_expert ||
        !aligned(num_tokens_per_expert, 4) || !grad_weight || !aligned(grad_weight, 16) ||
        !aligned(grad_bias, 4) || !aligned(workspace, 256))
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
    const Kind k = grad_kind_of(*p);
    const int64_t tiles = grad_tiles(*p, k);
    a.max_parts = max_parts(grad_depth(*p));
    a.stages = stages_of(grad_depth(*p));
    // (the number of tiles is known here: is any of them split?)
    const int64_t round = std::min<int64_t>(num_cus() * P::tile_groups(side_of(k)), tiles * a.max_parts);
    const bool join = a.max_parts > 1 &&
                      P::parts_of((int)(tiles % round), (int)round, a.max_parts, a.stages, side_of(k)) > 1;
    use_workspace(a, join ? workspace : nullptr);
    int rc = launch_kind<P::kWeightGrad>(k, a, tiles, s);
    if (rc == EPL_OK && grad_bias) {
        hipLaunchKernelGGL(P::bias_grad_kernel, dim3((unsigned)((a.N + 63) / 64), (unsigned)a.E),
                           dim3(P::kBiasThreads), 0, s, a, grad_bias);
        rc = launch_status();
    }
    return rc;
}

}  // extern "C"
