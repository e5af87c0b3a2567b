// Top-k routing: scores of each token's logits, the topk largest keys, their weights.
//
// One warp per token; expert j sits in lane j % 32.  A key is an order-preserving
// 32-bit integer (0: never chosen).  The topk-th largest of the 32 lanes' largest keys is a
// lower bound of the topk-th largest key, so the keys below it are out; the few that
// are left (about 1.5 topk) go to one lane each, which counts the candidates before its
// own: that count is its place in the result.  More than 32 candidates (ties) are taken by
// topk rounds of a warp maximum in place of that.
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
    // softmax weights that are normalised over the chosen need no other expert's score
    const bool late = !p.sigmoid && p.renormalize && !p.bias;
    if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = i * 32 + lane;
            const bool out = !(score[i] > -INFINITY);   // -infinity or NaN, and past the last expert
            score[i] = __frcp_rn(1.0f + expf(-score[i]));   // 1 / x, correctly rounded
            key[i] = out ? 0u : order_key(p.bias ? score[i] + p.bias[j] : score[i]);
        }
    } else {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = order_key(score[i]);
            if (late) continue;
            score[i] = key[i] ? expf(score[i] - top) : 0.0f;
            sum += score[i];
        }
        if (!late) {
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
        }
        denom = sum;
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key[i]) key[i] = order_key(score[i] / denom + p.bias[i * 32 + lane]);
        }
    }
    // the topk-th largest of the lanes' largest keys: a sort over the lanes, descending
    uint32_t bound = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) bound = max(bound, key[i]);
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int s = size >> 1; s > 0; s >>= 1) {
            const uint32_t other = __shfl_xor_sync(kFull, bound, s);
            const bool larger = ((lane & size) == 0) == ((lane & s) == 0);   // (lane & 32 is 0)
            bound = larger ? max(bound, other) : min(bound, other);
        }
    bound = max(__shfl_sync(kFull, bound, p.topk - 1), 1u);

    __shared__ uint32_t s_key[8][32];
    __shared__ float s_score[8][32];
    __shared__ int s_id[8][32];
    const int w = threadIdx.x >> 5;
    int count = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = key[i] >= bound;
        const uint32_t m = __ballot_sync(kFull, in);
        const int at = count + __popc(m & ((1u << lane) - 1u));
        if (in && at < 32) {
            s_key[w][at] = key[i];
            s_score[w][at] = score[i];
            s_id[w][at] = i * 32 + lane;
        }
        count += __popc(m);
    }
    __syncwarp();
    float chosen = 0.0f, mine = 0.0f;
    int my_id = -1, place = lane;
    if (count <= 32) {
        // candidates are in the order of their index
        const uint32_t k = lane < count ? s_key[w][lane] : 0u;
        int before = 0;
        for (int j = 0; j < count; ++j) {
            const uint32_t o = s_key[w][j];
            before += o > k || (o == k && j < lane);
        }
        const bool in = lane < count && before < p.topk;
        place = in ? before : 32;
        if (in) {
            my_id = s_id[w][lane];
            mine = late ? expf(s_score[w][lane] - top) : s_score[w][lane];
        }
        chosen = mine;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) chosen += __shfl_xor_sync(kFull, chosen, s);
        // slots that no expert is left for
        if (lane >= count && lane < p.topk) place = lane;
    } else {
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
            if (late) s = expf(s - top);
            chosen += s;
            if (lane == r) { my_id = win; mine = s; }
        }
    }
    if (place < p.topk) {
        if (p.renormalize) mine = mine / fmaxf(chosen, 1.17549435e-38f);
        else if (!p.sigmoid) mine = mine / denom;
        p.ids[static_cast<int64_t>(token) * p.topk + place] = my_id;
        p.weights[static_cast<int64_t>(token) * p.topk + place] = my_id < 0 ? 0.0f : mine * p.scale;
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
