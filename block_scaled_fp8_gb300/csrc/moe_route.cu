// Top-k routing: scores of each token's logits, the topk largest keys, their weights.
//
// One warp per token; expert j sits in lane j % 32.  A key is an order-preserving
// 32-bit integer (0: never chosen), so the warp's maximum and the lowest index among
// its holders are two integer reductions.  topk rounds, each removing its winner.
#include <cuda_bf16.h>

#include "dg_internal.h"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// Order-preserving map of a float to an unsigned integer; 0 for -infinity and NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and 0 are one key
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <int PER>
__global__ void __launch_bounds__(256) dg_moe_route_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const int token = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    grid_launch_dependents();
    grid_dependency_wait();
    if (token >= p.t) return;
    float score[PER];
    uint32_t key[PER];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = i * 32 + lane;
        float l = -INFINITY;
        if (j < p.experts)
            l = p.bf16 ? __uint_as_float(static_cast<uint32_t>(
                             static_cast<const uint16_t *>(p.logits)[token * p.ld + j]) << 16)
                       : static_cast<const float *>(p.logits)[token * p.ld + j];
        score[i] = l;
        if (l > top) top = l;
    }
    float denom = 1.0f;
    if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = i * 32 + lane;
            const bool out = !(score[i] > -INFINITY);   // -infinity or NaN, and past the last expert
            score[i] = 1.0f / (1.0f + expf(-score[i]));
            key[i] = out ? 0u : order_key(p.bias ? score[i] + p.bias[j] : score[i]);
        }
    } else {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = order_key(score[i]);
            score[i] = key[i] ? expf(score[i] - top) : 0.0f;
            sum += score[i];
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
        denom = sum;
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key[i]) key[i] = order_key(score[i] / denom + p.bias[i * 32 + lane]);
        }
    }
    float chosen = 0.0f, mine = 0.0f;
    int my_id = -1;
    for (int r = 0; r < p.topk; ++r) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key[i]);
        const uint32_t m = __reduce_max_sync(kFull, best);
        if (m == 0) break;
        int at = 1 << 30;
        float s = 0.0f;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] == m) { at = i * 32 + lane; s = score[i]; }
        const int win = __reduce_min_sync(kFull, at);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * 32 + lane == win) key[i] = 0u;
        s = __shfl_sync(kFull, s, win & 31);
        chosen += s;
        if (lane == r) { my_id = win; mine = s; }
    }
    if (lane < p.topk) {
        if (p.renormalize) mine = mine / fmaxf(chosen, 1.17549435e-38f);
        else if (!p.sigmoid) mine = mine / denom;
        p.ids[static_cast<int64_t>(token) * p.topk + lane] = my_id;
        p.weights[static_cast<int64_t>(token) * p.topk + lane] = my_id < 0 ? 0.0f : mine * p.scale;
    }
}

template <int PER>
cudaError_t launch(const RouteParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((p.t + 7) / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dg_moe_route_kernel<PER>, p);
}

}  // namespace

cudaError_t launch_moe_route(const RouteParams &p, cudaStream_t stream) {
    if (p.experts <= 32) return launch<1>(p, stream);
    if (p.experts <= 64) return launch<2>(p, stream);
    if (p.experts <= 128) return launch<4>(p, stream);
    if (p.experts <= 256) return launch<8>(p, stream);
    if (p.experts <= 512) return launch<16>(p, stream);
    return launch<32>(p, stream);
}

}  // namespace dg
