// Few-row products and the MoE layer for few tokens: plain CUDA-core kernels, one
// warp per row of weights, FP32 sums.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dg_internal.h"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float scale_of(uint32_t byte) {   // 2^(byte - 127)
    return byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7FFFFFFFu)
                                                                  : __uint_as_float(byte << 23);
}

__device__ __forceinline__ float e2m1(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float v = e == 0 ? 0.5f * m : __uint_as_float(((e + 126u) << 23) | (m << 22));
    return c & 8u ? -v : v;
}

// Weights k..k+3 of one row, without their scale.
template <bool FP4>
__device__ __forceinline__ void load4(const uint8_t *row, int k, float (&w)[4]) {
    if constexpr (FP4) {
        const uint32_t c = *reinterpret_cast<const uint16_t *>(row + k / 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e2m1((c >> (4 * j)) & 15u);
    } else {
        const uint32_t c = *reinterpret_cast<const uint32_t *>(row + k);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = __half2float(__half(__nv_cvt_fp8_to_halfraw((c >> (8 * j)) & 255u, __NV_E4M3)));
    }
}

// Scale of weights k.. of one row; sf points at the row's word of slice 0, ld words per slice.
template <bool FP4>
__device__ __forceinline__ float scale_at(const uint32_t *sf, int64_t ld, int k) {
    const int g = FP4 ? k / 32 : k / 128;
    return scale_of((sf[(g >> 2) * ld] >> (8 * (g & 3))) & 255u);
}

// sum_k w[k] x[k] over the warp (x: bf16 or FP32)
template <bool FP4, typename X>
__device__ __forceinline__ float dot(const uint8_t *row, const uint32_t *sf, int64_t ld, const X *x, int k, int lane) {
    float acc = 0.0f;
    for (int i = lane * 4; i < k; i += 128) {
        float w[4];
        load4<FP4>(row, i, w);
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = static_cast<float>(x[i + j]);
            part += w[j] * v + (v - v);   // a non-finite activation gives NaN, whatever its weight
        }
        acc += part * scale_at<FP4>(sf, ld, i);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) acc += __shfl_xor_sync(kFull, acc, s);
    return acc;
}

template <bool FP4, bool F32>
__global__ void __launch_bounds__(256) dg_few_gemv_kernel(const FewParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= p.n) return;
    for (int m = 0; m < p.m; ++m) {
        float v = dot<FP4>(p.b + n * p.ldb, p.sfb + n, (p.n + 3) / 4 * 4,
                           reinterpret_cast<const __nv_bfloat16 *>(p.a + m * p.lda), p.k, lane);
        if (lane != 0) continue;
        if constexpr (F32) {
            if (p.c) v += static_cast<const float *>(p.c)[m * p.ldc + n];
            static_cast<float *>(p.d)[m * p.ldd + n] = v;
        } else {
            if (p.c) v += static_cast<float>(static_cast<const __nv_bfloat16 *>(p.c)[m * p.ldc + n]);
            static_cast<__nv_bfloat16 *>(p.d)[m * p.ldd + n] = __float2bfloat16_rn(v);
        }
    }
}

template <bool FP4>
__global__ void __launch_bounds__(256) dg_moe_up_kernel(const LayerParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int pair = blockIdx.y;
    const int e = p.ids[pair];
    if (e >= p.experts && p.status && threadIdx.x == 0) atomicOr(p.status, DG_DEV_BAD_GROUP);
    if (j >= p.i || e < 0 || e >= p.experts) return;
    const int64_t row_bytes = FP4 ? p.h / 2 : p.h;
    const int64_t slices = FP4 ? p.h / 128 : (p.h + 511) / 512;
    const int64_t ld = 2 * p.i;
    const uint8_t *w = p.w1 + e * ld * row_bytes;
    const uint32_t *sf = p.sf1 + e * slices * ld;
    const __nv_bfloat16 *x = reinterpret_cast<const __nv_bfloat16 *>(p.x + pair / p.topk * p.ldx);
    const float g = dot<FP4>(w + j * row_bytes, sf + j, ld, x, p.h, lane);
    const float u = dot<FP4>(w + (p.i + j) * row_bytes, sf + p.i + j, ld, x, p.h, lane);
    if (lane == 0) p.act[static_cast<int64_t>(pair) * p.i + j] = g / (1.0f + expf(-g)) * u;
}

template <bool FP4>
__global__ void __launch_bounds__(256) dg_moe_down_kernel(const LayerParams p) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = blockIdx.y;
    if (n >= p.h) return;
    const int64_t row_bytes = FP4 ? p.i / 2 : p.i;
    const int64_t slices = FP4 ? p.i / 128 : (p.i + 511) / 512;
    float y = p.c ? static_cast<float>(reinterpret_cast<const __nv_bfloat16 *>(p.c)[t * p.ldc + n]) : 0.0f;
    for (int j = 0; j < p.topk; ++j) {
        const int pair = t * p.topk + j;
        const int e = p.ids[pair];
        if (e < 0 || e >= p.experts) continue;
        y += p.weights[pair] * dot<FP4>(p.w2 + (static_cast<int64_t>(e) * p.h + n) * row_bytes,
                                        p.sf2 + e * slices * p.h + n, p.h,
                                        p.act + static_cast<int64_t>(pair) * p.i, p.i, lane);
    }
    if (lane == 0) reinterpret_cast<__nv_bfloat16 *>(p.y)[t * p.ldy + n] = __float2bfloat16_rn(y);
}

}  // namespace

cudaError_t launch_few_gemv(const FewParams &p, int num_sms, cudaStream_t stream) {
    const dim3 grid((p.n + 7) / 8);
    if (p.fp4)
        p.f32 ? dg_few_gemv_kernel<true, true><<<grid, 256, 0, stream>>>(p)
              : dg_few_gemv_kernel<true, false><<<grid, 256, 0, stream>>>(p);
    else
        p.f32 ? dg_few_gemv_kernel<false, true><<<grid, 256, 0, stream>>>(p)
              : dg_few_gemv_kernel<false, false><<<grid, 256, 0, stream>>>(p);
    host_set_last_config(1, 8, 1, static_cast<int>(grid.x), 3, 1);
    return cudaGetLastError();
}

cudaError_t launch_moe_layer(const LayerParams &p, int num_sms, cudaStream_t stream) {
    const dim3 up((p.i + 7) / 8, p.t * p.topk), down((p.h + 7) / 8, p.t);
    if (p.fp4) {
        dg_moe_up_kernel<true><<<up, 256, 0, stream>>>(p);
        dg_moe_down_kernel<true><<<down, 256, 0, stream>>>(p);
    } else {
        dg_moe_up_kernel<false><<<up, 256, 0, stream>>>(p);
        dg_moe_down_kernel<false><<<down, 256, 0, stream>>>(p);
    }
    host_set_last_config(1, 8, 1, static_cast<int>(up.x * up.y), 4, 2);
    return cudaGetLastError();
}

}  // namespace dg
