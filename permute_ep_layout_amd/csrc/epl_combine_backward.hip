// The gradient of the combine (epl_combine_backward, include/epl.h): kernel
// and host side.
//
// With y[t] = sum_k w[t,k] v[o[t,k]]:
//     d v[o[t,k]] = w[t,k] * d y[t]            (one rounding to bf16)
//     d w[t,k]    = sum_h d y[t,h] * v[o[t,k],h]   (binary32)
// One pass over the expert rows: each is read for its dot product and its
// gradient written while the token's d y sits in registers, so the bytes are
// those of one read and one write of every routed row, which is the bound:
// 4096 tokens, top-8, hidden 7168 move 0.999 GB in 191 us, 5.2 TB/s (a plain
// copy of 2 GiB: 4.9).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epl.h"

namespace epl_combine_grad {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kSlots = 8;       // slots that share a pass over d y

struct Args {
    const void *dy;
    const __bf16 *v;
    const int32_t *oi;
    const float *w;
    __bf16 *dv;
    float *dw;
    uint32_t *status;
    int64_t T, rows;
    int K, H;
};

template <bool BF16>
__device__ __forceinline__ void load_dy(const void *p, int64_t at, float (&d)[8])
{
    if (BF16) {
        const bf16x8 r = *reinterpret_cast<const bf16x8 *>(static_cast<const __bf16 *>(p) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d[i] = (float)r[i];
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + 4);
        d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w;
        d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
    }
}

// WAVES waves a token share its columns; their partial dot products are
// added in wave order through LDS. STREAM: rows past the caches, in and out.
template <bool BF16, int WAVES, bool STREAM>
__global__ __launch_bounds__(WAVES * 64) void kernel(Args a)
{
    __shared__ float part[WAVES][kSlots];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        for (int k0 = 0; k0 < a.K; k0 += kSlots) {
            int64_t row[kSlots];
            float w[kSlots], dot[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                const int k = k0 + s;
                int64_t o = k < a.K ? a.oi[t * a.K + k] : -1;
                if (o >= a.rows) {
                    if (a.status && tid == 0)
                        atomicOr(a.status, 4u);          // an output_index beyond the rows
                    o = -1;
                }
                row[s] = o;
                w[s] = o >= 0 ? a.w[t * a.K + k] : 0.0f;
                dot[s] = 0.0f;
            }
            for (int h = tid * 8; h < a.H; h += WAVES * 512) {
                float d[8];
                load_dy<BF16>(a.dy, t * a.H + h, d);
                bf16x8 v[kSlots];
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (row[s] >= 0) {
                        const auto *at = reinterpret_cast<const bf16x8 *>(a.v + row[s] * a.H + h);
                        v[s] = STREAM ? __builtin_nontemporal_load(at) : *at;
                    }
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (row[s] < 0)
                        continue;
                    bf16x8 g;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[s] = fmaf(d[i], (float)v[s][i], dot[s]);
                        g[i] = (__bf16)(w[s] * d[i]);
                    }
                    auto *at = reinterpret_cast<bf16x8 *>(a.dv + row[s] * a.H + h);
                    if (STREAM)
                        __builtin_nontemporal_store(g, at);
                    else
                        *at = g;
                }
            }
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                for (int m = 32; m > 0; m >>= 1)
                    dot[s] += __shfl_xor(dot[s], m);
            if (lane == 0)
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    part[wave][s] = dot[s];
            __syncthreads();
            if (tid < kSlots && k0 + tid < a.K) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < WAVES; ++i)
                    sum += part[i][tid];
                a.dw[t * a.K + k0 + tid] = sum;
            }
            __syncthreads();
        }
    }
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace epl_combine_grad

extern "C" int epl_combine_backward(const epl_problem *p, int grad_type, const void *grad_y,
                                    const uint16_t *expert_out, int64_t expert_rows,
                                    const int32_t *output_index, const float *topk_weights,
                                    uint16_t *grad_rows, float *grad_weights, void *workspace,
                                    void *stream)
{
    namespace C = epl_combine_grad;
    if (epl_validate(p) != EPL_OK || (grad_type != EPL_OUT_F32 && grad_type != EPL_OUT_BF16))
        return EPL_EINVAL;
    if (expert_rows < 0 || (workspace && !C::aligned(workspace, 256)))
        return EPL_EINVAL;
    if (p->num_tokens == 0)
        return EPL_OK;
    if (!grad_y || !C::aligned(grad_y, 16) || !output_index || !C::aligned(output_index, 4) ||
        !topk_weights || !C::aligned(topk_weights, 4) || !grad_weights ||
        !C::aligned(grad_weights, 4) ||
        (expert_rows > 0 && (!expert_out || !C::aligned(expert_out, 16) || !grad_rows ||
                             !C::aligned(grad_rows, 16))))
        return EPL_EINVAL;
    C::Args a{};
    a.dy = grad_y;
    a.v = reinterpret_cast<const __bf16 *>(expert_out);
    a.oi = output_index;
    a.w = topk_weights;
    a.dv = reinterpret_cast<__bf16 *>(grad_rows);
    a.dw = grad_weights;
    a.status = static_cast<uint32_t *>(workspace);      // the header's first word
    a.T = p->num_tokens;
    a.rows = expert_rows;
    a.K = p->num_topk;
    a.H = p->hidden;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)std::min<int64_t>(a.T, 1 << 20));
    auto launch = [&](auto kernel, int waves) {
        hipLaunchKernelGGL(kernel, grid, dim3(waves * 64), 0, s, a);
    };
    const bool bf16 = grad_type == EPL_OUT_BF16;
    // A wave a token where a row is two passes of 512 columns at most; more
    // share longer rows: 8 where the rows stay in the caches (64 tokens, top-8,
    // 7168 columns: 8.5 us, against 8.9 with 4), and 4 that pass them by where
    // they do not (4096 tokens: 192 us, 5.2 TB/s, against 205 through them).
    const bool stream_rows = a.T * a.K * (int64_t)a.H * 2 > (int64_t(128) << 20);
    if (a.H <= 1024)
        stream_rows ? (bf16 ? launch(C::kernel<true, 1, true>, 1) : launch(C::kernel<false, 1, true>, 1))
                    : (bf16 ? launch(C::kernel<true, 1, false>, 1) : launch(C::kernel<false, 1, false>, 1));
    else if (stream_rows)
        bf16 ? launch(C::kernel<true, 4, true>, 4) : launch(C::kernel<false, 4, true>, 4);
    else
        bf16 ? launch(C::kernel<true, 8, false>, 8) : launch(C::kernel<false, 8, false>, 8);
    return hipGetLastError() == hipSuccess ? EPL_OK : EPL_EHIP;
}
