// Top-k routing: scores of each token's logits, the topk largest keys, their weights.
//
// One warp per token.  Bound by the instructions that it issues (E logits are read
// once, 4 E bytes a token), so no expert that cannot be chosen is worked on:
//  - every lane takes the largest approximate key of its experts (the logit for softmax,
//    else the score by one approximate tanh, within kCoarse);
//  - the topk-th largest of the 32 lanes' values (topk rounds of a maximum over the lanes),
//    less twice the error, is a lower bound of the topk-th largest key; the experts not
//    below it are candidates (about 1.2 topk);
//  - each candidate goes to one lane, which computes its score and key in full and counts
//    the candidates before it: its place in the result.
// More than 32 candidates of a sigmoid (scores close to 1) are looked for once more with its
// approximation by exponential and reciprocal, within kFine; where they are still more (ties),
// topk rounds of a maximum over all keys take them.
//
// Measured, calls in a row in a graph: 32768 x 256, top 8 of sigmoid + bias, FP32 17.9 us (33.5 MB
// of logits take 5.0 us; 500 instructions a token fill 79 % of the issue slots), softmax
// without bias 15.4 us, 4099 x 128, top 6 of softmax, bf16 4.7 us, one token 2.2 us (a launch).
#include <cuda_bf16.h>

#include "dg_internal.h"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
// Above twice the errors of the approximate sigmoids.  1/2 + tanh(x / 2) / 2: tanh.approx is
// within 2^-11 of its value.  1 / (1 + e): the exponential's argument is off by 2^-24 of
// itself and exponential and reciprocal by 2^-22, which moves it by at most 1e-6.
constexpr float kCoarse = 6e-4f, kFine = 4e-6f;

// Order-preserving map of a float to an unsigned integer; 0 for -infinity and NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and 0 are one key
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

__device__ __forceinline__ float tanh_approx(float x) {
    float r;
    asm("tanh.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max_over_lanes(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// x of the lane `d` below added, in lanes that have one
__device__ __forceinline__ int add_from_below(int x, int d) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 v;\n\t"
        "shfl.sync.up.b32 v|p, %0, %1, 0, 0xffffffff;\n\t"
        "@p add.s32 %0, %0, v;\n\t}"
        : "+r"(x)
        : "r"(d));
    return x;
}

__device__ __forceinline__ float sigmoid_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-x)));
    return r;
}

// Lane l holds experts PER l .. PER l + PER - 1.
template <int PER, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(256) dg_moe_route_kernel(const RouteParams p) {
    constexpr int VEC = PER < 4 ? PER : 4;
    const int lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int token = blockIdx.x * 8 + w;
    __shared__ __align__(16) float s_x[8][32 * PER];
    __shared__ __align__(16) uint32_t s_key[8][32];
    __shared__ int s_id[8][32];
    grid_launch_dependents();
    grid_dependency_wait();
    if (token >= p.t) return;

    float x[PER];      // logits; -infinity where none
    const char *row = static_cast<const char *>(p.logits) + token * p.ld * (BF16 ? 2 : 4);
#pragma unroll
    for (int i0 = 0; i0 < PER; i0 += VEC) {
        const int j0 = lane * PER + i0;
        if (VEC == 4 && p.vec) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i0 + i] = -INFINITY;
            if (j0 < p.experts) {
                if constexpr (BF16) {
                    const uint2 v = __ldcg(reinterpret_cast<const uint2 *>(row + 2 * j0));
                    const uint32_t u[2] = {v.x, v.y};
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        x[i0 + i] = __uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
                } else {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(row + 4 * j0));
                    const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < VEC; ++i) x[i0 + i] = u[i];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[i0 + i] = -INFINITY;
                if (j0 + i < p.experts)
                    x[i0 + i] =
                        BF16 ? __uint_as_float(static_cast<uint32_t>(__ldcg(
                                   reinterpret_cast<const uint16_t *>(row) + j0 + i)) << 16)
                             : __ldcg(reinterpret_cast<const float *>(row) + j0 + i);
            }
        }
    }
    if constexpr (VEC == 4) {
#pragma unroll
        for (int i = 0; i < PER; i += 4)
            *reinterpret_cast<float4 *>(&s_x[w][lane * PER + i]) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) s_x[w][lane * PER + i] = x[i];
    }
    float top = -INFINITY, denom = 1.0f;
    // softmax weights that are normalised over the chosen need no other expert's score
    const bool late = !SIGMOID && p.renormalize;
    if constexpr (!SIGMOID) {
#pragma unroll
        for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
        if (!late || p.bias) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (x[i] > -INFINITY) sum += expf(x[i] - top);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
            denom = sum;
        }
    }
    auto bias_of = [&](int j) { return p.bias ? __ldg(p.bias + j) : 0.0f; };
    // approximate keys; -infinity or NaN for what is never chosen
    float approx[PER], low = x[0];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (SIGMOID) approx[i] = 0.5f;
        else approx[i] = p.bias ? expf(x[i] - top) / denom : x[i];
        low = fminf(low, x[i]);
    }
    if (p.bias) {
        const float *bias = p.bias + lane * PER;
#pragma unroll
        for (int i0 = 0; i0 < PER; i0 += VEC) {
            if (VEC == 4 && p.vec_bias) {
                if (lane * PER + i0 >= p.experts) break;
                const float4 v = __ldg(reinterpret_cast<const float4 *>(bias + i0));
                const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < VEC; ++i) approx[i0 + i] += u[i];
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (lane * PER + i0 + i < p.experts) approx[i0 + i] += __ldg(bias + i0 + i);
            }
        }
    }
    if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < PER; ++i) approx[i] = fmaf(0.5f, tanh_approx(0.5f * x[i]), approx[i]);
    }
    float slack = SIGMOID ? kCoarse : p.bias ? kFine : 0.0f;
    uint32_t hits;
    int at, count;
    while (true) {
        if (low == -INFINITY) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (x[i] == -INFINITY) approx[i] = -INFINITY;
        }
        __syncwarp();
        float best = -INFINITY, bound = INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = fmaxf(best, approx[i]);
        // the topk-th largest of the lanes' largest (lower where some are equal)
        for (int r = 0; r < p.topk; ++r) {
            bound = max_over_lanes(best);
            if (best == bound) best = -INFINITY;
        }
        if (slack != 0.0f && fabsf(bound) < INFINITY)
            bound -= slack + fabsf(bound) * 2.4e-7f;   // (and the key's own rounding)
        bound = fmaxf(bound, -3.402823466e38f);
        hits = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (approx[i] >= bound) hits |= 1u << i;
        at = __popc(hits);
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) at = add_from_below(at, s);
        count = __shfl_sync(kFull, at, 31);
        if (!SIGMOID || count <= 32 || slack == kFine) break;
        slack = kFine;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            approx[i] = sigmoid_approx(x[i]) + (lane * PER + i < p.experts ? bias_of(lane * PER + i) : 0.0f);
    }
    float score = 0.0f, chosen = 0.0f;
    int id = -1, place = lane;
    if (count <= 32) {
        // the candidates, in the order of their index
        for (at -= __popc(hits); hits; hits &= hits - 1u) s_id[w][at++] = lane * PER + __ffs(hits) - 1;
        __syncwarp();
        uint32_t key = 0;
        if (lane < count) {
            id = s_id[w][lane];
            const float l = s_x[w][id];
            score = SIGMOID ? sigmoid(l) : expf(l - top);
            if (!SIGMOID && !late) score /= denom;
            if constexpr (SIGMOID) key = order_key(score + bias_of(id));
            else key = order_key(p.bias ? expf(l - top) / denom + bias_of(id) : l);
        }
        s_key[w][lane] = key;
        __syncwarp();
        int before = 0;
        for (int j = 0; j < count; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4 *>(&s_key[w][j]);
            before += o.x > key;
            before += o.y > key;
            before += o.z > key;
            before += o.w > key;
        }
        // (a key that is NaN is 0; candidates beyond the topk have no place)
        const bool valid = key != 0u;
        const int valids = __popc(__ballot_sync(kFull, valid));
        if (__popc(__reduce_or_sync(kFull, valid ? 1u << before : 0u)) != valids) {
            for (int j = 0; j < lane; ++j) before += s_key[w][j] == key;   // of equal keys the earlier comes first
            __syncwarp();
        }
        const bool in = valid && before < p.topk;
        place = in ? before : 32;
        if (!in) {
            id = -1;
            score = 0.0f;
        }
        if (valids < p.topk) {   // the slots that no expert is left for go to the idle lanes
            const uint32_t placed = __ballot_sync(kFull, in);
            if (!in) place = __popc(placed) + __popc(~placed & ((1u << lane) - 1u));
        }
        chosen = score;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) chosen += __shfl_xor_sync(kFull, chosen, s);
    } else {
        uint32_t key[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = 0u;
            if (!(x[i] > -INFINITY)) continue;
            if constexpr (SIGMOID) key[i] = order_key(sigmoid(x[i]) + bias_of(lane * PER + i));
            else key[i] = order_key(p.bias ? expf(x[i] - top) / denom + bias_of(lane * PER + i) : x[i]);
        }
        __syncwarp();
        for (int r = 0; r < p.topk; ++r) {
            uint32_t high = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) high = max(high, key[i]);
            const uint32_t m = __reduce_max_sync(kFull, high);
            if (m == 0) break;
            int first = 1 << 30;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (key[i] == m) first = lane * PER + i;
            const int win = __reduce_min_sync(kFull, first);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane * PER + i == win) key[i] = 0u;
            const float l = s_x[w][win];
            float s = SIGMOID ? sigmoid(l) : expf(l - top);
            if (!SIGMOID && !late) s /= denom;
            chosen += s;
            if (lane == r) { id = win; score = s; }
        }
    }
    if (place < p.topk) {
        if (p.renormalize) score /= fmaxf(chosen, 1.17549435e-38f);
        const int64_t out = static_cast<int64_t>(token) * p.topk + place;
        p.ids[out] = id;
        p.weights[out] = id < 0 ? 0.0f : score * p.scale;
    }
}

template <int PER, bool BF16, bool SIGMOID>
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
    return cudaLaunchKernelEx(&cfg, dg_moe_route_kernel<PER, BF16, SIGMOID>, p);
}

template <int PER>
cudaError_t launch_per(const RouteParams &p, cudaStream_t stream) {
    if (p.bf16) return p.sigmoid ? launch<PER, true, true>(p, stream) : launch<PER, true, false>(p, stream);
    return p.sigmoid ? launch<PER, false, true>(p, stream) : launch<PER, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_moe_route(const RouteParams &params, cudaStream_t stream) {
    RouteParams p = params;
    // rows of whole aligned groups of 4 experts are read a group at a time
    p.vec = p.experts % 4 == 0 && p.ld % 4 == 0 &&
            reinterpret_cast<uintptr_t>(p.logits) % (p.bf16 ? 8 : 16) == 0;
    p.vec_bias = p.experts % 4 == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
    if (p.experts <= 32) return launch_per<1>(p, stream);
    if (p.experts <= 64) return launch_per<2>(p, stream);
    if (p.experts <= 128) return launch_per<4>(p, stream);
    if (p.experts <= 256) return launch_per<8>(p, stream);
    if (p.experts <= 512) return launch_per<16>(p, stream);
    return launch_per<32>(p, stream);
}

}  // namespace dg
