// libepl.so host side of the router: argument checks and launches of
// epl_route and epl_route_backward (include/epl.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "epl.h"
#include "epl_router_kernels.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launch_status() { return hipGetLastError() == hipSuccess ? EPL_OK : EPL_EHIP; }

bool router_ok(const epl_router *p)
{
    if (!p || p->reserved != 0)
        return false;
    if (p->num_experts < 1 || p->num_experts > epl_router_k::kMaxExperts)
        return false;
    if (p->num_topk < 1 || p->num_topk > epl_router_k::kMaxTopk || p->num_topk > p->num_experts)
        return false;
    if (p->num_tokens < 0 || p->num_tokens > INT32_MAX / p->num_topk)
        return false;
    if (p->score != EPL_SCORE_SOFTMAX && p->score != EPL_SCORE_SIGMOID)
        return false;
    if (p->logits_type != EPL_OUT_F32 && p->logits_type != EPL_OUT_BF16)
        return false;
    if (p->num_groups < 1 || p->num_groups > epl_router_k::kMaxGroups ||
        p->num_experts % p->num_groups != 0)
        return false;
    if (p->topk_groups < 1 || p->topk_groups > p->num_groups || p->group_top < 1 ||
        p->group_top > 2)
        return false;
    if ((int64_t)p->topk_groups * (p->num_experts / p->num_groups) < p->num_topk)
        return false;
    if (p->renormalize != 0 && p->renormalize != 1)
        return false;
    return std::isfinite(p->scale);
}

// Rows that 16-byte loads can read: each starts on a multiple of 16 bytes.
bool vector_rows(const epl_router &p, const void *a, const void *b)
{
    return p.num_experts % (p.logits_type == EPL_OUT_BF16 ? 8 : 4) == 0 && aligned(a, 16) &&
           aligned(b, 16);
}

}  // namespace

extern "C" {

int epl_router_validate(const epl_router *p) { return router_ok(p) ? EPL_OK : EPL_EINVAL; }

int epl_route(const epl_router *p, const void *logits, const float *bias,
              const uint8_t *token_mask, int64_t *topk_idx, float *topk_weights, void *stream)
{
    if (!router_ok(p))
        return EPL_EINVAL;
    const size_t size = p->logits_type == EPL_OUT_BF16 ? 2 : 4;
    if (bias && !aligned(bias, 4))
        return EPL_EINVAL;
    if (p->num_tokens == 0)
        return EPL_OK;
    if (!logits || !aligned(logits, size) || !topk_idx || !aligned(topk_idx, 8) || !topk_weights ||
        !aligned(topk_weights, 4))
        return EPL_EINVAL;
    namespace R = epl_router_k;
    R::Args a{};
    a.logits = logits;
    a.bias = bias;
    a.mask = token_mask;
    a.idx = topk_idx;
    a.w = topk_weights;
    a.T = p->num_tokens;
    a.K = p->num_topk;
    a.E = p->num_experts;
    a.G = p->topk_groups == p->num_groups ? 1 : p->num_groups;    // all groups: no choice of groups
    a.topk_groups = p->topk_groups;
    a.group_top = p->group_top;
    a.softmax = p->score == EPL_SCORE_SOFTMAX;
    a.renorm = p->renormalize != 0;
    a.bf16 = p->logits_type == EPL_OUT_BF16;
    a.need_scores = bias || (a.G > 1 && a.group_top == 2);
    a.vec = vector_rows(*p, logits, logits);
    a.bias_vec = aligned(bias, 16);
    a.scale = p->scale;
    hipStream_t s = static_cast<hipStream_t>(stream);

    // pieces of 8 experts; groups must be a power of two of whole pieces
    const int pieces = (a.E + 7) / 8;
    const int per = a.G > 1 && (a.E / a.G) % 8 == 0 ? a.E / a.G / 8 : 0;
    const bool groups_fit = a.G == 1 || (per > 0 && (per & (per - 1)) == 0);
    a.per_log = per > 0 ? 31 - __builtin_clz((unsigned)per) : 0;
    auto launch = [&](auto kernel, int L) {
        const int tok = R::kThreads / L;
        hipLaunchKernelGGL(kernel, dim3((unsigned)((a.T + tok - 1) / tok)), dim3(R::kThreads), 0, s,
                           a);
        return launch_status();
    };
    if (a.K <= 8 && groups_fit && a.T <= INT32_MAX / 64) {
        // Lanes a token: few, so that a wave holds many tokens and shares its
        // instructions among them, where there are tokens enough to fill the
        // GPU; with few tokens as many lanes as there are pieces, the
        // shortest path for one token.
        const bool many = a.T > 4096;
        auto order = [&](auto o) {
            constexpr R::Order O = decltype(o)::value;
            if (pieces <= 8 && per <= 8)
                return launch(R::route_kernel<8, 1, O>, 8);
            if (pieces <= 16 && per <= 16)
                return launch(R::route_kernel<16, 1, O>, 16);
            if (pieces <= 32 && per <= 8 && many)
                return launch(R::route_kernel<8, 4, O>, 8);
            if (pieces <= 32 && per <= 32)
                return launch(R::route_kernel<32, 1, O>, 32);
            if (pieces <= 64 && per <= 64)
                return launch(R::route_kernel<64, 1, O>, 64);
            return launch(R::route_kernel<64, 4, O>, 64);
        };
        if (pieces <= 256 && per <= 64)
            return !a.need_scores ? order(std::integral_constant<R::Order, R::kLogits>{})
                   : a.softmax    ? order(std::integral_constant<R::Order, R::kSoftmax>{})
                                  : order(std::integral_constant<R::Order, R::kSigmoid>{});
    }
    hipLaunchKernelGGL(R::route_any_kernel, dim3((unsigned)std::min<int64_t>(a.T, 1 << 16)),
                       dim3(64), 0, s, a);
    return launch_status();
}

int epl_route_backward(const epl_router *p, const void *logits, const int64_t *topk_idx,
                       const float *grad_weights, void *grad_logits, void *stream)
{
    if (!router_ok(p))
        return EPL_EINVAL;
    const size_t size = p->logits_type == EPL_OUT_BF16 ? 2 : 4;
    if (p->num_tokens == 0)
        return EPL_OK;
    if (!logits || !aligned(logits, size) || !topk_idx || !aligned(topk_idx, 8) || !grad_weights ||
        !aligned(grad_weights, 4) || !grad_logits || !aligned(grad_logits, size))
        return EPL_EINVAL;
    namespace R = epl_router_k;
    R::GradArgs a{};
    a.K = p->num_topk;
    a.E = p->num_experts;
    a.softmax = p->score == EPL_SCORE_SOFTMAX;
    a.renorm = p->renormalize != 0;
    a.bf16 = p->logits_type == EPL_OUT_BF16;
    a.vec = vector_rows(*p, logits, grad_logits);
    a.scale = p->scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int pieces = (a.E + 7) / 8;
    auto launch = [&](auto kernel, int L) {
        const int tok = R::kThreads / L;
        // at most 2^30 work-items a launch (a loop over tokens in the kernel
        // took 27.7 us instead of 25.9 for 65536 x 256 logits)
        const int64_t most = (int64_t)tok << 22, T = p->num_tokens;
        for (int64_t t0 = 0; t0 < T; t0 += most) {
            a.T = std::min(T - t0, most);
            a.logits = static_cast<const char *>(logits) + t0 * a.E * size;
            a.idx = topk_idx + t0 * a.K;
            a.g = grad_weights + t0 * a.K;
            a.out = static_cast<char *>(grad_logits) + t0 * a.E * size;
            hipLaunchKernelGGL(kernel, dim3((unsigned)((a.T + tok - 1) / tok)), dim3(R::kThreads),
                               0, s, a);
        }
        return launch_status();
    };
    if (pieces <= 8)
        return launch(R::route_grad_kernel<8, 1>, 8);
    if (pieces <= 16)
        return launch(R::route_grad_kernel<16, 1>, 16);
    if (pieces <= 32)
        return launch(R::route_grad_kernel<32, 1>, 32);
    if (pieces <= 64)
        return launch(R::route_grad_kernel<64, 1>, 64);
    return launch(R::route_grad_kernel<64, 4>, 64);
}

}  // extern "C"
