// Newton-Schulz orthogonalisation of a matrix (the update of an orthogonalising optimiser):
// X0 = G / (|G|_F + eps), then `steps` times
//     A = X X^T,   B = b A + c A A,   X <- a X + B X
// for X with the short side as its rows (a tall G is transposed on the way in and out).
//
// All three products are FP16 x FP16 -> FP32 on CTA pairs (tcgen05 cta_group::2, kind::f16):
// 256x256 tiles, operands by TMA with 128-byte swizzle in stages of 64 K, two accumulators in
// TMEM, so that a tile's epilogue runs beside the next tile's MMAs.  Roles: warp 0 producer,
// warp 1 MMA issuer (leader), warps 2-9 epilogue.
//
// Numbers: the operands are FP16 (11 bits) scaled by 2^12, which keeps the iteration's values
// (|X| <= 1.3, |A| <= 1.5, |B| <= 3 with the usual coefficients) below 2^14 and their small ones
// normal down to 2^-26.  X itself is kept as two FP16 planes, high and low (22 bits): the high plane
// is the operand, and a X + B X is formed from both.  With X rounded to 11 bits in each step its
// error is multiplied by a = 3.4 a step in every direction that G hardly has, and comes to 4e-2 of
// the result for a gradient with a decaying spectrum; with the low plane it is 1e-3 or less
// (bf16's own rounding of the result: 1.7e-3).  Sums are FP32, the norm FP64.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "dg_internal.h"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr float kScale = 4096.0f;          // of all FP16 planes
constexpr int kTile = 256;                 // rows and columns of a pair tile
constexpr int kKBlock = 64;                // K of a stage: 128 bytes
constexpr int kStages = 6;
constexpr int kStageBytes = 2 * 128 * 128; // A and B: 128 rows of 128 bytes each
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kSmem = 1024 + kStages * kStageBytes + 256;

// ------------------------------------------------------------------ norm and split

// Sum of squares of a matrix, as partial sums of CTAs: three FP32 accumulators (values below 2^-40,
// above 2^40, between, the outer ones scaled), so that no square over- or underflows, then FP64.
template <bool BF16>
__global__ void __launch_bounds__(256) dg_ns_norm_kernel(const __grid_constant__ NsParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t batch = blockIdx.y;
    const char *g = static_cast<const char *>(p.g) + batch * p.g_batch * (BF16 ? 2 : 4);
    double total = 0.0;
    float mid = 0.f, big = 0.f, small = 0.f;
    auto add = [&](float v) {
        const float m = fabsf(v);
        if (m >= 0x1p-40f && m <= 0x1p40f) mid = fmaf(v, v, mid);
        else if (m < 0x1p-40f) { const float s = v * 0x1p80f; small = fmaf(s, s, small); }
        else { const float s = v * 0x1p-70f; big = fmaf(s, s, big); }   // (NaN here too)
    };
    auto flush = [&]() {
        total += static_cast<double>(mid) + static_cast<double>(small) * 0x1p-160 + static_cast<double>(big) * 0x1p140;
        mid = big = small = 0.f;
    };
    // dense matrices are one long row; a CTA takes segments of a row
    const int64_t len = p.dense ? static_cast<int64_t>(p.rows) * p.cols : p.cols;
    const int64_t rows = p.dense ? 1 : p.rows;
    constexpr int64_t kSeg = 8192;
    const int64_t segs = (len + kSeg - 1) / kSeg;
    for (int64_t s = blockIdx.x; s < rows * segs; s += gridDim.x) {
        const int64_t row = s / segs, c0 = (s - row * segs) * kSeg;
        const int64_t n = len - c0 < kSeg ? len - c0 : kSeg;
        const char *at = g + (row * p.ldg + c0) * (BF16 ? 2 : 4);
        constexpr int V = BF16 ? 8 : 4;
        if ((reinterpret_cast<uintptr_t>(at) & 15u) == 0) {
            const int64_t nv = n / V;
#pragma unroll 4
            for (int64_t i = threadIdx.x; i < nv; i += 256) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(at) + i);
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (BF16) {
                        add(__uint_as_float(x[j] << 16));
                        add(__uint_as_float(x[j] & 0xFFFF0000u));
                    } else {
                        add(__uint_as_float(x[j]));
                    }
                }
            }
            const int64_t i = nv * V + threadIdx.x;
            if (i < n)
                add(BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(at)[i]) << 16)
                         : reinterpret_cast<const float *>(at)[i]);
        } else {
            for (int64_t i = threadIdx.x; i < n; i += 256)
                add(BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(at)[i]) << 16)
                         : reinterpret_cast<const float *>(at)[i]);
        }
        flush();
    }
    __shared__ double part[8];
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) total += part[w];
        p.partial[batch * p.num_partial + blockIdx.x] = total;
    }
}

// X0 as high and low planes [lo][ld], transposed where G is tall; tiles of 64x64 through shared memory.
template <bool BF16>
__global__ void __launch_bounds__(256) dg_ns_split_kernel(const __grid_constant__ NsParams p) {
    __shared__ float tile[64][65];
    __shared__ double sum;
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t batch = blockIdx.z;
    // every CTA adds the partial sums in the same order
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int i = threadIdx.x; i < p.num_partial; i += 32) s += p.partial[batch * p.num_partial + i];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (threadIdx.x == 0) sum = s;
    }
    __syncthreads();
    // 2^12 / (norm + eps) in two factors, so that neither leaves FP32's range
    const double norm = sqrt(sum) + static_cast<double>(p.eps);
    int e = 0;
    const double mant = norm > 0.0 ? frexp(static_cast<double>(kScale) / norm, &e) : 0.0;
    const int e1 = e / 2;
    const float f1 = static_cast<float>(ldexp(1.0, e1)), f2 = static_cast<float>(ldexp(mant, e - e1));
    const char *g = static_cast<const char *>(p.g) + batch * p.g_batch * (BF16 ? 2 : 4);
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of G
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int r = r0 + i / 64, c = c0 + i % 64;
        float v = 0.f;
        if (r < p.rows && c < p.cols) {
            const int64_t at = static_cast<int64_t>(r) * p.ldg + c;
            v = BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(g)[at]) << 16)
                     : reinterpret_cast<const float *>(g)[at];
        }
        tile[i / 64][i % 64] = v * f1 * f2;
    }
    __syncthreads();
    const bool tall = p.rows > p.cols;
    const int x0 = tall ? c0 : r0, y0 = tall ? r0 : c0;     // of X
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int r = i / 32, c = 2 * (i % 32);
        if (x0 + r >= p.lo || y0 + c >= p.hi) continue;
        const float a = tall ? tile[c][r] : tile[r][c], b = tall ? tile[c + 1][r] : tile[r][c + 1];
        const __half2 h = __floats2half2_rn(a, b);
        const __half2 l = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
        const int64_t at = (batch * p.lo + x0 + r) * p.ldx + y0 + c;
        *reinterpret_cast<__half2 *>(p.xh[0] + at) = h;      // (ld is even: the pair past the end is padding)
        *reinterpret_cast<__half2 *>(p.xl + at) = l;
    }
}

// ------------------------------------------------------------------ products

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

enum NsMode : int { kNsGram = 0, kNsPoly = 1, kNsUpdate = 2, kNsLast = 3 };

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 half2_values(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// 16 consecutive FP16 values (rows are padded to whole chunks of 16).
__device__ __forceinline__ void load16(const uint16_t *at, uint32_t (&w)[8]) {
    const uint4 a = __ldcg(reinterpret_cast<const uint4 *>(at)), b = __ldcg(reinterpret_cast<const uint4 *>(at) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// MODE kNsGram: D = A; kNsPoly: D = b A + c A A; kNsUpdate: X planes of a X + B X; kNsLast: the same
// to the bf16 output.  The first two are [lo][lo] products of K-major operands; the others take X as
// the MN-major operand ([K][N], N contiguous).
template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    dg_ns_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ NsParams p, const int k) {
    constexpr bool B_MN = MODE >= kNsUpdate;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *smem_a = smem, *smem_b = smem + kStages * 16384;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);
    uint64_t *full_bar = bars;                   // [kStages] leader: both CTAs' stages landed
    uint64_t *empty_bar = full_bar + kStages;    // [kStages] both: MMAs done with the stage
    uint64_t *tfull_bar = empty_bar + kStages;   // [2] both: accumulator complete
    uint64_t *tempty_bar = tfull_bar + 2;        // [2] leader: both epilogues drained
    uint64_t *drain_bar = tempty_bar + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    WaitCtl ctl{abort_flag, p.status, p.timeout_ns};
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int pair_id = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const int rows = p.lo, cols = MODE >= kNsUpdate ? p.hi : p.lo;
    const int tm = (rows + kTile - 1) / kTile, tn = (cols + kTile - 1) / kTile;
    const int per = tm * tn, num_tiles = per * p.batch;
    const int nkb = (k + kKBlock - 1) / kKBlock;

    if (warp == 0) {
        if (lane < 2 * kStages + 5) mbar_init(bars + lane, bars + lane >= tempty_bar && bars + lane < tempty_bar + 2 ? 2 * kEpiWarps : 1);
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
        if (lane == 0) {
            tma_prefetch_desc(&tm_a);
            tma_prefetch_desc(&tm_b);
        }
    }
    grid_launch_dependents();
    grid_dependency_wait();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;

    // tile t: (batch, m, n), the m tiles of a column of tiles first
    auto locate = [&](int t, int &b, int &m0, int &n0) {
        b = t / per;
        const int r = t - b * per;
        m0 = (r % tm) * kTile;
        n0 = (r / tm) * kTile;
    };

    if (warp == 0) {
        const uint32_t leader_full = mapa_shared(smem_u32(full_bar), 0);
        int slot = 0;
        uint32_t phase = 0, issued = 0;
        bool drop = (p.debug_flags & DG_DEBUG_DROP_ONE_LOAD) && pair_id == 0 && MODE == kNsGram;
        for (int t = pair_id; t < num_tiles; t += num_pairs) {
            int b, m0, n0;
            locate(t, b, m0, n0);
            for (int kb = 0; kb < nkb; ++kb) {
                if (!mbar_wait_warp(&empty_bar[slot], phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto prod_done;
                if (drop) {
                    drop = false;   // diagnostic: leave this stage empty
                } else {
                    if (elect_one()) {
                        const uint32_t fb = leader_full + slot * 8;
                        if (leader) mbar_arrive_expect_tx(&full_bar[slot], 2 * kStageBytes);
                        tma_load_3d_pair(smem_a + slot * 16384, &tm_a, fb, kb * kKBlock, m0 + rank * 128, b);
                        if constexpr (B_MN) {
                            // 64 columns (one swizzle atom) x 64 K rows a box
                            tma_load_3d_pair(smem_b + slot * 16384, &tm_b, fb, n0 + rank * 128, kb * kKBlock, b);
                            tma_load_3d_pair(smem_b + slot * 16384 + 8192, &tm_b, fb, n0 + rank * 128 + 64, kb * kKBlock, b);
                        } else {
                            tma_load_3d_pair(smem_b + slot * 16384, &tm_b, fb, kb * kKBlock, n0 + rank * 128, b);
                        }
                    }
                    __syncwarp();
                    issued |= 1u << slot;
                }
                if (++slot == kStages) { slot = 0; phase ^= 1; }
            }
        }
    prod_done:
        if (lane == 0 && leader)
            for (int s = 0; s < kStages; ++s)
                if (issued & (1u << s)) mbar_wait_drain(&full_bar[s], s < slot ? phase : phase ^ 1, ctl);
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            int slot = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            // FP16 x FP16 -> FP32, M = 256, N = 256, B MN-major where X is
            constexpr uint32_t idesc = (1u << 4) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24) | (B_MN ? 1u << 16 : 0u);
            const uint64_t a0 = make_desc_kmajor_sw128(smem_u32(smem_a));
            // (MN-major: the two 64-column atoms 8192 bytes apart, 8 K rows 1024)
            const uint64_t b0 = B_MN ? make_smem_desc(smem_u32(smem_b), 8192, 1024, kSwizzle128B)
                                     : make_desc_kmajor_sw128(smem_u32(smem_b));
            constexpr uint64_t kStepB = B_MN ? (2048 >> 4) : 2;   // 16 K: 16 rows, or 32 bytes along a row
            for (int t = pair_id; t < num_tiles; t += num_pairs) {
                if (!mbar_wait_cluster_warp(&tempty_bar[acc], acc_phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto mma_done;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + acc * kTile;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!mbar_wait_warp(&full_bar[slot], phase, ctl, DG_DEV_TIMEOUT)) goto mma_done;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t a = a0 + slot * (16384 >> 4), b = b0 + slot * (16384 >> 4);
#pragma unroll
                        for (int s = 0; s < 4; ++s) mma_f16_pair(d, a + 2 * s, b + kStepB * s, idesc, (kb | s) != 0);
                        tc_commit_pair(&empty_bar[slot], 0x3);
                    }
                    __syncwarp();
                    if (++slot == kStages) { slot = 0; phase ^= 1; }
                }
                if (elect_one()) tc_commit_pair(&tfull_bar[acc], 0x3);
                __syncwarp();
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
        mma_done:
            if (elect_one()) {
                tc_commit_pair(drain_bar, 0x1);
                mbar_wait(drain_bar, 0, ctl, DG_DEV_TIMEOUT);
            }
            __syncwarp();
        }
    } else {
        const uint32_t ew = warp - 2, quad = warp & 3, half = ew >> 2;
        const uint32_t leader_tempty = mapa_shared(smem_u32(tempty_bar), 0);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int t = pair_id; t < num_tiles; t += num_pairs) {
            int b, m0, n0;
            locate(t, b, m0, n0);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull_bar[acc], acc_phase, ctl, DG_DEV_TIMEOUT))) break;
            tc_fence_after_sync();
            const int row = m0 + rank * 128 + static_cast<int>(quad) * 32 + static_cast<int>(lane);
            const int col0 = n0 + static_cast<int>(half) * 128;
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem_base + ((quad * 32) << 16) + acc * kTile + half * 128 + c, v);
                tmem_ld_wait();
                reg_fence16(v);
                const int col = col0 + c;
                if (row >= rows || col >= cols) continue;
                float f[16];
                if constexpr (MODE == kNsGram) {
                    // 2^24 X X^T -> 2^12 A
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]) * (1.0f / kScale);
                } else if constexpr (MODE == kNsPoly) {
                    uint32_t a[8];
                    load16(p.a + (static_cast<int64_t>(b) * p.lo + row) * p.lda + col, a);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 x = half2_values(a[i]);
                        f[2 * i] = fmaf(p.cb, x.x, p.cc * (1.0f / kScale) * __uint_as_float(v[2 * i]));
                        f[2 * i + 1] = fmaf(p.cb, x.y, p.cc * (1.0f / kScale) * __uint_as_float(v[2 * i + 1]));
                    }
                } else {
                    const int64_t at = (static_cast<int64_t>(b) * p.lo + row) * p.ldx + col;
                    uint32_t xh[8], xl[8];
                    load16(p.xh[0] + at, xh);
                    load16(p.xl + at, xl);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 h = half2_values(xh[i]), l = half2_values(xl[i]);
                        f[2 * i] = fmaf(p.ca, h.x + l.x, (1.0f / kScale) * __uint_as_float(v[2 * i]));
                        f[2 * i + 1] = fmaf(p.ca, h.y + l.y, (1.0f / kScale) * __uint_as_float(v[2 * i + 1]));
                    }
                }
                if constexpr (MODE == kNsLast) {
                    uint16_t *out = p.out + b * p.out_batch;
                    const bool tall = p.rows > p.cols;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (col + i >= cols) break;
                        const __nv_bfloat16 o = __float2bfloat16_rn(f[i] * (1.0f / kScale));
                        out[tall ? static_cast<int64_t>(col + i) * p.ldo + row : static_cast<int64_t>(row) * p.ldo + col + i] =
                            *reinterpret_cast<const uint16_t *>(&o);
                    }
                } else {
                    uint32_t o[8], l[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[i] = half2_bits(f[2 * i], f[2 * i + 1]);
                        if constexpr (MODE == kNsUpdate) {
                            const float2 h = half2_values(o[i]);
                            l[i] = half2_bits(f[2 * i] - h.x, f[2 * i + 1] - h.y);
                        }
                    }
                    const int64_t ld = MODE == kNsUpdate ? p.ldx : p.lda;
                    const int64_t at = (static_cast<int64_t>(b) * p.lo + row) * ld + col;
                    uint16_t *dst = MODE == kNsGram ? p.a : MODE == kNsPoly ? p.b : p.xh[1];
                    uint4 *d = reinterpret_cast<uint4 *>(dst + at);
                    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
                    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
                    if constexpr (MODE == kNsUpdate) {
                        d = reinterpret_cast<uint4 *>(p.xl + at);
                        d[0] = make_uint4(l[0], l[1], l[2], l[3]);
                        d[1] = make_uint4(l[4], l[5], l[6], l[7]);
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(leader_tempty + acc * 8);
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// 3-D map of planes [batch][rows][ld] of FP16: boxes of 64 elements (128 bytes) x box_rows.
bool encode_plane(CUtensorMap *map, const uint16_t *base, int64_t cols, int64_t rows, int64_t ld, int64_t batch,
                  uint32_t box_rows) {
    TensorMapEncodeFn fn = host_encode();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld * rows) * 2};
    const cuuint32_t box[3] = {kKBlock, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Co-resident CTA pairs on the current device, at most num_sms / 2.
template <int MODE>
int max_pairs(int num_sms) {
    static std::mutex mu;
    static int cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int &v = cache[dev];
    if (v == 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&v, dg_ns_gemm_kernel<MODE>, &cfg) != cudaSuccess) v = 0;
    }
    return v * 2 > num_sms ? num_sms / 2 : v;
}

template <int MODE>
cudaError_t launch_product(const NsParams &p, const CUtensorMap &a, const CUtensorMap &b, int k, int num_sms,
                           cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(dg_ns_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = up(p.lo, kTile) / kTile * (up(MODE >= kNsUpdate ? p.hi : p.lo, kTile) / kTile) * p.batch;
    const int pairs = max_pairs<MODE>(num_sms);
    if (pairs <= 0) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(2 * static_cast<int>(tiles < pairs ? tiles : pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dg_ns_gemm_kernel<MODE>, a, b, p, k);
}

cudaError_t launch_simple(void (*kernel)(NsParams), dim3 grid, const NsParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

constexpr int kMaxPartial = 304;

}  // namespace

// Two high planes, the low plane, A and B, and the norm's partial sums; rows of whole 64-element
// (128-byte) lines.
int64_t ns_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    const int64_t lo = rows < cols ? rows : cols, hi = rows < cols ? cols : rows;
    return batch * (2 * lo * (3 * up(hi, 64) + 2 * up(lo, 64)) + 8 * kMaxPartial);
}

cudaError_t launch_newton_schulz(NsParams p, int steps, bool bf16, int num_sms, cudaStream_t stream, int *launches) {
    p.lo = p.rows < p.cols ? p.rows : p.cols;
    p.hi = p.rows < p.cols ? p.cols : p.rows;
    p.ldx = up(p.hi, 64);
    p.lda = up(p.lo, 64);
    uint8_t *w = static_cast<uint8_t *>(p.workspace);
    auto take = [&w](int64_t bytes) { uint8_t *at = w; w += bytes; return reinterpret_cast<uint16_t *>(at); };
    const int64_t plane = 2 * p.batch * p.lo * p.ldx, square = 2 * static_cast<int64_t>(p.batch) * p.lo * p.lda;
    p.xh[0] = take(plane);
    p.xh[1] = take(plane);
    p.xl = take(plane);
    p.a = take(square);
    p.b = take(square);
    p.partial = reinterpret_cast<double *>(w);
    p.dense = p.ldg == p.cols;
    const int64_t segs = p.dense ? (static_cast<int64_t>(p.rows) * p.cols + 8191) / 8192 : p.rows * ((p.cols + 8191ll) / 8192);
    p.num_partial = static_cast<int>(segs < kMaxPartial ? segs : kMaxPartial);   // (by the matrix alone, as its sum's order)
    cudaError_t e = launch_simple(bf16 ? dg_ns_norm_kernel<true> : dg_ns_norm_kernel<false>, dim3(p.num_partial, p.batch), p, stream);
    if (e != cudaSuccess) return e;
    e = launch_simple(bf16 ? dg_ns_split_kernel<true> : dg_ns_split_kernel<false>,
                      dim3((p.cols + 63) / 64, (p.rows + 63) / 64, p.batch), p, stream);
    *launches = 2 + 3 * steps;
    CUtensorMap ma, mb, mx[2], mxn[2];
    for (int i = 0; i < 2; ++i)
        if (!encode_plane(&mx[i], p.xh[i], p.hi, p.lo, p.ldx, p.batch, 128) ||
            !encode_plane(&mxn[i], p.xh[i], p.hi, p.lo, p.ldx, p.batch, kKBlock))
            return cudaErrorInvalidValue;
    if (!encode_plane(&ma, p.a, p.lo, p.lo, p.lda, p.batch, 128) || !encode_plane(&mb, p.b, p.lo, p.lo, p.lda, p.batch, 128))
        return cudaErrorInvalidValue;
    int cur = 0;
    uint16_t *planes[2] = {p.xh[0], p.xh[1]};
    for (int s = 0; s < steps && e == cudaSuccess; ++s) {
        p.xh[0] = planes[cur];
        p.xh[1] = planes[cur ^ 1];
        e = launch_product<kNsGram>(p, mx[cur], mx[cur], p.hi, num_sms, stream);
        if (e == cudaSuccess) e = launch_product<kNsPoly>(p, ma, ma, p.lo, num_sms, stream);
        if (e == cudaSuccess)
            e = s + 1 < steps ? launch_product<kNsUpdate>(p, mb, mxn[cur], p.lo, num_sms, stream)
                              : launch_product<kNsLast>(p, mb, mxn[cur], p.lo, num_sms, stream);
        p.debug_flags = 0;
        cur ^= 1;
    }
    return e;
}

}  // namespace dg
