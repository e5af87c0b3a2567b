// Newton-Schulz orthogonalisation of a matrix (the update of an orthogonalising optimiser):
// X0 = G / (|G|_F + eps), then `steps` times
//     A = X X^T,   B = b A + c A A,   X <- a X + B X
// for X with the short side as its rows (a tall G is transposed on the way in and out).
//
// All three products are FP16 x FP16 -> FP32 on CTA pairs (tcgen05 cta_group::2, kind::f16):
// 256x256 tiles (or 128 or 64 columns where tiles are few), operands by TMA with 128-byte swizzle in
// stages of 64 K, two accumulators in TMEM, so that a tile's epilogue runs beside the next tile's
// MMAs.  Roles: warp 0 producer, warp 1 MMA issuer (leader), warps 2-9 epilogue.
// Bound by: large matrices, the card's power limit (4x2048x7168: 1.42 ms in bursts of ten calls, 1.46
// PFLOP/s of the products that are run, and 1.61 to 1.67 ms when repeated for long, at 1.45 GHz; the update's
// planes, 470 MB a step, add 0.05 ms a step); middle ones, the pairs that a product's tiles leave idle
// (2x2112x1536: a step's 42, 42 and 108 tiles on 76 pairs take 105 K-block times where an even share is 66); small
// ones, the chain of a phase, 3.3 us and 0.2 us a K-block (64x64: 4 us a phase).
//
// Numbers: the operands are FP16 (11 bits) scaled by 2^12, which keeps the iteration's values
// (|X| <= 1.3, |A| <= 1.5, |B| <= 3 with the usual coefficients) below 2^14 and their small ones
// normal down to 2^-26.  X itself is kept as two FP16 planes, high and low (22 bits): the high plane
// is the operand, and a X + B X is formed from both.  With X rounded to 11 bits in each step its
// error is multiplied by a = 3.4 a step in every direction that G hardly has, and comes to 4e-2 of
// the result for a gradient with a decaying spectrum; with the low plane it is 1e-3 or less where the
// short side is 250 or more (bf16's own rounding of the result: 1.7e-3).  B times what the high plane leaves
// out of X, strong directions mixed into weak ones, falls with the square root of the short side, so that
// small matrices need it: up to a short side of 192 the update's product takes the low plane too, twice its
// K-blocks (error with 8 strong directions, 64x64: 3.4e-3 without, 7e-4 with; 200x200: 1.1e-3 without; singular
// values over four decades, 4x4: 2.2e-2 and 1.5e-3.  64x64: 63.3 us without, 64.0 with; 700x40x64: 287 and
// 292; 128x2048: 103 and 105; 250x1000, which goes without: 93 and 97).
// Sums are FP32, the norm's partial sums FP64.
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
// Ring: stages of 128 rows of A and up to as much of B; as many as fit, 5 of 32 KB with tiles of 256
// columns, 6 of 24 KB with narrower ones, whose K-blocks are bound by the bytes in flight
constexpr int kMaxStages = 6;
constexpr int kRingBytes = 5 * 32768;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
// Epilogue: an epilogue warp's 32 rows x 128 columns of a tile in chunks of 32 columns; a chunk
// passes through one of two slots of two boxes (32 rows of 64 bytes, 64-byte swizzle)
constexpr int kBoxBytes = 32 * 64;
constexpr int kSlotBytes = 2 * kBoxBytes;
constexpr int kEpiBytes = kEpiWarps * 2 * kSlotBytes;
constexpr int kSmem = 1024 + kRingBytes + kEpiBytes + 128 * kEpiWarps + 512;

// A stage: A's 16 KB, then B's largest part.
__host__ __device__ constexpr int ring_stage_bytes(int bn_sym, int bn_update) {
    const int b_sym = bn_sym * 64, b_update = bn_update == kTile ? 16384 : 8192;
    return 16384 + (b_sym > b_update ? b_sym : b_update);
}
__host__ __device__ constexpr int ring_stages(int bn_sym, int bn_update) {
    const int n = kRingBytes / ring_stage_bytes(bn_sym, bn_update);
    return n < kMaxStages ? n : kMaxStages;
}

// ------------------------------------------------------------------ norm and split

template <bool BF16>
__device__ __forceinline__ float g_value(const char *g, int64_t at) {
    return BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(g)[at]) << 16)
                : reinterpret_cast<const float *>(g)[at];
}

// Sum of squares of a matrix, as partial sums of CTAs.  A thread adds the squares of its 32 values of
// a segment in FP32, beside their largest magnitude; where that lies outside 2^-40 .. 2^40 (0 aside), the
// segment is added again with its values scaled into the range, so that no square over- or
// underflows.  The segments' sums are FP32 for 32 of them, then FP64 (64-bit sums throughout
// would take most of the kernel's time: a few a clock and SM).
template <bool BF16>
__global__ void __launch_bounds__(256) dg_ns_norm_kernel(const __grid_constant__ NsParams p) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t batch = blockIdx.y;
    const char *g = static_cast<const char *>(p.g) + batch * p.g_batch * (BF16 ? 2 : 4);
    double total = 0.0;
    float run = 0.f;
    // dense matrices are one long row; a CTA takes segments of a row
    const int64_t len = p.dense ? static_cast<int64_t>(p.rows) * p.cols : p.cols;
    const int64_t rows = p.dense ? 1 : p.rows;
    constexpr int kSeg = 8192, V = BF16 ? 8 : 4;
    const int64_t segs = (len + kSeg - 1) / kSeg;
    int since = 0;
    for (int64_t s = blockIdx.x; s < rows * segs; s += gridDim.x) {
        const int64_t row = segs == 1 ? s : s / segs, c0 = (s - row * segs) * kSeg;
        const int n = static_cast<int>(len - c0 < kSeg ? len - c0 : kSeg);
        const char *at = g + (row * p.ldg + c0) * (BF16 ? 2 : 4);
        const bool vec = (reinterpret_cast<uintptr_t>(at) & 15u) == 0;
        float sum, amax;
        auto segment = [&](float scale) {
            sum = amax = 0.f;
            auto add = [&](float v) {
                v *= scale;
                sum = fmaf(v, v, sum);
                amax = fmaxf(amax, fabsf(v));
            };
            // (V values a thread in their order, whether the address allows a load of 16 bytes or not)
            if (vec) {
#pragma unroll 8
                for (int i = threadIdx.x; i < n / V; i += 256) {
                    const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(at) + i);
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
            } else {
#pragma unroll 4
                for (int i = threadIdx.x; i < n / V; i += 256)
#pragma unroll
                    for (int j = 0; j < V; ++j) add(g_value<BF16>(at, i * V + j));
            }
            for (int i = n / V * V + threadIdx.x; i < n; i += 256) add(g_value<BF16>(at, i));
        };
        segment(1.0f);
        if (amax > 0x1p40f) {
            segment(0x1p-70f);
            total += static_cast<double>(sum) * 0x1p140;
        } else if (amax < 0x1p-40f && amax > 0.f) {
            segment(0x1p80f);
            total += static_cast<double>(sum) * 0x1p-160;
        } else {
            run += sum;   // (a NaN stays one)
        }
        if (++since == 32) {
            total += run;
            run = 0.f;
            since = 0;
        }
    }
    __shared__ double part[8];
    // (FP32 over a warp: five more roundings of 2^-24)
    for (int o = 16; o > 0; o >>= 1) run += __shfl_xor_sync(0xFFFFFFFFu, run, o);
    if (__any_sync(0xFFFFFFFFu, total != 0.0))
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = total + run;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0.0;
        for (int w = 0; w < 8; ++w) total += part[w];
        p.partial[batch * p.num_partial + blockIdx.x] = total;
    }
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// 2^12 / (sqrt(s) + eps) in two factors, so that neither leaves FP32's range: FP32 arithmetic on
// significands beside integer exponents (a few roundings of 2^-24, all of X alike).  With a 64-bit square
// root and division, a chain of its own in every CTA of the split, a call took 1 us more (250x1000:
// 92.0 us against 90.9).  s: 0, 2^-298 .. 2^300, infinite or NaN.
__device__ __forceinline__ void inverse_norm(double s, float eps, float &f1, float &f2) {
    const uint32_t hi = static_cast<uint32_t>(__double2hiint(s));
    if (!(hi < 0x7FF00000u)) {   // infinite: 0, NaN: NaN
        f1 = 1.0f;
        f2 = kScale / static_cast<float>(s);
        return;
    }
    // sqrt(s) = r 2^es, eps = q 2^ee, r and q in [1, 2) or 0
    const int k = static_cast<int>(hi >> 20) - 1023, es = s == 0.0 ? -1000 : k >> 1;
    const int top = static_cast<int>((hi & 0xFFFFFu) | static_cast<uint32_t>(1023 + (k & 1)) << 20);
    const float r = s == 0.0 ? 0.0f : sqrtf(static_cast<float>(__hiloint2double(top, __double2loint(s))));
    const int ee = eps == 0.0f ? -1000 : eps < 0x1p-126f ? -126 : static_cast<int>(__float_as_uint(eps) >> 23) - 127;
    if (es < -500 && ee < -500) {   // 0: X is 0
        f1 = f2 = 0.0f;
        return;
    }
    const int e = es > ee ? es : ee;   // (eps infinite: 128, and 1 / norm 0)
    const float norm = (es - e > -64 ? r * pow2(es - e) : 0.0f) +
                       (ee - e > -64 ? eps * pow2(-(ee >> 1)) * pow2((ee >> 1) - e) : 0.0f);
    const int to = 12 - e, e1 = to >> 1;
    f1 = pow2(e1);
    f2 = pow2(to - e1) / norm;
}

// The factors of a matrix.  Every CTA adds the partial sums in the same order.
__device__ __forceinline__ void norm_factors(const NsParams &p, int64_t batch, float &f1, float &f2) {
    __shared__ float factors[2];
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int i = threadIdx.x; i < p.num_partial; i += 32) s += p.partial[batch * p.num_partial + i];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (threadIdx.x == 0) inverse_norm(s, p.eps, factors[0], factors[1]);
    }
    // (the products' grid counter and abort word, which follow in the stream)
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 2) p.sync[threadIdx.x] = 0u;
    __syncthreads();
    f1 = factors[0];
    f2 = factors[1];
}

// Two values as high and low FP16 pairs.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const __half2 l = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// X0 as high and low planes [lo][ldx].  A wide G row by row, 8 values a thread (16-byte loads where
// the rows allow them); a tall G transposed through 64x64 tiles in shared memory.
template <bool BF16, bool TALL>
__global__ void __launch_bounds__(256) dg_ns_split_kernel(const __grid_constant__ NsParams p) {
    __shared__ float tile[TALL ? 64 : 1][65];
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t batch = blockIdx.z;
    float f1, f2;
    norm_factors(p, batch, f1, f2);
    const char *g = static_cast<const char *>(p.g) + batch * p.g_batch * (BF16 ? 2 : 4);
    if constexpr (!TALL) {
        constexpr int kRows = 8;   // of G, 2048 columns each
        const int c = static_cast<int>(blockIdx.x) * 2048 + static_cast<int>(threadIdx.x) * 8;
        const bool vec = (reinterpret_cast<uintptr_t>(g) & 15u) == 0 && p.ldg % (BF16 ? 8 : 4) == 0 && c + 8 <= p.cols;
        if (c >= p.cols) return;
#pragma unroll 4
        for (int i = 0; i < kRows; ++i) {
            const int r = static_cast<int>(blockIdx.y) * kRows + i;
            if (r >= p.rows) break;
            const int64_t at = static_cast<int64_t>(r) * p.ldg + c;
            float v[8];
            if (vec) {
                const uint4 *q = reinterpret_cast<const uint4 *>(g + at * (BF16 ? 2 : 4));
                const uint4 a = __ldcg(q);
                const uint32_t x[4] = {a.x, a.y, a.z, a.w};
                if constexpr (BF16) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[2 * j] = __uint_as_float(x[j] << 16);
                        v[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
                    }
                } else {
                    const uint4 b = __ldcg(q + 1);
                    const uint32_t y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j] = __uint_as_float(x[j]);
                        v[4 + j] = __uint_as_float(y[j]);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = c + j < p.cols ? g_value<BF16>(g, at + j) : 0.f;
            }
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split2(v[2 * j] * f1 * f2, v[2 * j + 1] * f1 * f2, h[j], l[j]);
            const int64_t to = (batch * p.lo + r) * p.ldx + c;   // (rows are padded to whole 64s)
            *reinterpret_cast<uint4 *>(p.xh[0] + to) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(p.xl + to) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    } else {
        // kTiles tiles of 64x64 down a column of tiles: the factors are worked out once a CTA
        constexpr int kTiles = 4, V = BF16 ? 8 : 4;
        const int c0 = blockIdx.x * 64;                         // of G
        const bool vec = (reinterpret_cast<uintptr_t>(g) & 15u) == 0 && p.ldg % V == 0 && c0 + 64 <= p.cols;
        for (int i = 0; i < kTiles; ++i) {
            const int r0 = (static_cast<int>(blockIdx.y) * kTiles + i) * 64;
            if (r0 >= p.rows) break;
            if (vec) {
                constexpr int kPer = 64 / V;
#pragma unroll
                for (int q = threadIdx.x; q < 64 * kPer; q += 256) {
                    const int r = q / kPer, c = q % kPer * V;
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (r0 + r < p.rows)
                        x = __ldcg(reinterpret_cast<const uint4 *>(
                            g + (static_cast<int64_t>(r0 + r) * p.ldg + c0 + c) * (BF16 ? 2 : 4)));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (BF16) {
                            tile[r][c + 2 * j] = __uint_as_float(w[j] << 16) * f1 * f2;
                            tile[r][c + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * f1 * f2;
                        } else {
                            tile[r][c + j] = __uint_as_float(w[j]) * f1 * f2;
                        }
                    }
                }
            } else {
#pragma unroll 8
                for (int q = threadIdx.x; q < 64 * 64; q += 256) {
                    const int r = r0 + q / 64, c = c0 + q % 64;
                    tile[q / 64][q % 64] =
                        r < p.rows && c < p.cols ? g_value<BF16>(g, static_cast<int64_t>(r) * p.ldg + c) * f1 * f2 : 0.f;
                }
            }
            __syncthreads();
#pragma unroll
            for (int q = threadIdx.x; q < 64 * 8; q += 256) {
                const int r = q / 8, c = 8 * (q % 8);           // of X's tile
                if (c0 + r >= p.lo || r0 + c >= p.hi) continue;
                uint32_t h[4], l[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) split2(tile[c + 2 * j][r], tile[c + 2 * j + 1][r], h[j], l[j]);
                const int64_t to = (batch * p.lo + c0 + r) * p.ldx + r0 + c;
                *reinterpret_cast<uint4 *>(p.xh[0] + to) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(p.xl + to) = make_uint4(l[0], l[1], l[2], l[3]);
            }
            __syncthreads();
        }
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
__device__ __forceinline__ float2 half2_values(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// MODE kNsGram: D = A; kNsPoly: D = b A + c A A; kNsUpdate: X planes of a X + B X; kNsLast: the same
// to the bf16 output.  The first two are [lo][lo] products of K-major operands and symmetric: the
// tiles on and above the diagonal are computed, and those above it stored twice, once transposed.
// The others take X as the MN-major operand ([K][N], N contiguous).
//
// The diagonals of A and B are kept apart in FP32 and are 0 in the FP16 matrices: with A = D + R,
// A A = D D + D R + R D + R R, and B X = diag(B) X + (rest) X.  Near convergence X X^T is close to
// the identity, so that the diagonal holds most of A and B, and its rounding to 11 bits most of
// the error: with it in FP32 the result's error is about half (noise 512x512: 7e-4 against 1.5e-3
// of its norm).
//
// The epilogue's own operands (A; the planes of X) come by TMA into the boxes that the results go
// out from, two chunks ahead.
//
// All products of all steps are one cooperative launch: each is a phase, and a phase's tiles wait for all
// tiles of the one before (a counter of finished tiles in the workspace, polled by the producer
// warps, with a limit).  As launches of their own they cost 7.5 us each however small (64x64, five
// steps: 127 us against 67).
// Several matrices may go in two groups with a counter each, the second a phase behind: while one
// group waits for its phase's last tiles, the other has work, and the few tiles of a symmetric
// product run beside the many of an update (choose_tiles).
struct NsMaps {
    CUtensorMap xk[2], xn[2];   // X's high planes along K (128 rows a box), and as [K][N]
    CUtensorMap xln;            // the low plane as [K][N]
    CUtensorMap a, b;           // A, B along K
    CUtensorMap xkb[2], ab;     // X and A as the second operand of a symmetric product: bn_sym / 2 rows a box
    CUtensorMap xh[2], xl, ea, eb, out;   // boxes of the epilogue
};

// Short side up to which an update's product goes over both planes of X.  (Its tiles have one row then: the pair
// that computes a tile is the only one that reads these columns of the low plane, which its epilogue replaces.)
constexpr int kLowPlaneSide = 192;
static_assert(kLowPlaneSide <= kTile, "the low plane is read and replaced by the same pair");

// K-blocks of a product.
__host__ __device__ inline int ns_kblocks(int mode, int lo, int hi) {
    const int n = ((mode == kNsGram ? hi : lo) + kKBlock - 1) / kKBlock;
    return mode >= kNsUpdate && lo <= kLowPlaneSide ? 2 * n : n;
}

// What a phase works on.
struct NsPhase {
    int mode, step, cols, bn, tm, tn, per, num_tiles, nkb;
    int b0;      // the group's first matrix
    int first;   // this pair's first tile
};

// Phase i of group g, or of no tiles where it has no such phase.
__device__ __forceinline__ NsPhase ns_shape(const NsParams &p, int i, int g) {
    NsPhase f;
    f.step = i / 3;
    f.mode = i % 3;
    if (f.mode == kNsUpdate && f.step + 1 == p.steps) f.mode = kNsLast;
    const bool sym = f.mode < kNsUpdate;
    f.cols = sym ? p.lo : p.hi;
    f.bn = sym ? p.bn_sym : p.bn_update;
    f.tm = (p.lo + kTile - 1) / kTile;
    f.tn = (f.cols + f.bn - 1) / f.bn;
    // symmetric: the column tiles of diagonal block q (kTile / bn of them) have row tiles 0..q
    const int r = kTile / f.bn, q = f.tn / r;
    f.per = sym ? r * (q * (q + 1) / 2) + (f.tn - r * q) * (q + 1) : f.tm * f.tn;
    f.b0 = g == 0 ? 0 : p.group0;
    f.num_tiles = i < 0 || i >= 3 * p.steps ? 0 : f.per * (g == 0 ? p.group0 : p.batch - p.group0);
    f.nkb = ns_kblocks(f.mode, p.lo, p.hi);
    return f;
}

// The phase that group g has in turn `turn`: its phase turn - g.  The second group's tiles go on from
// the pair after the first group's last.
__device__ __forceinline__ NsPhase ns_phase(const NsParams &p, int turn, int g, int pair_id, int num_pairs) {
    NsPhase f = ns_shape(p, turn - g, g);
    f.first = pair_id;
    if (g > 0) {
        f.first = pair_id - ns_shape(p, turn, 0).num_tiles % num_pairs;
        if (f.first < 0) f.first += num_pairs;
    }
    return f;
}

// What group g's counter has come to when its phases before phase i are finished: both CTAs of a
// tile's pair count it.
__device__ __forceinline__ uint32_t ns_finished(const NsParams &p, int i, int g) {
    const uint32_t sym = ns_shape(p, 0, g).num_tiles, update = ns_shape(p, 2, g).num_tiles, r = i % 3;
    return 2u * (i / 3 * (2u * sym + update) + r * sym);
}

// Tile t of a phase: (batch, m, n), the m tiles of a column of tiles first
__device__ __forceinline__ void ns_locate(const NsPhase &f, int t, int &b, int &m0, int &n0) {
    b = t / f.per;
    const int i = t - b * f.per;
    b += f.b0;
    if (f.mode < kNsUpdate) {
        const int r = kTile / f.bn, h = i / r;   // q(q+1)/2 <= h < (q+1)(q+2)/2
        int q = static_cast<int>((sqrtf(8.0f * static_cast<float>(h) + 1.0f) - 1.0f) * 0.5f);
        while (q * (q + 1) / 2 > h) --q;
        while ((q + 1) * (q + 2) / 2 <= h) ++q;
        const int in = i - r * (q * (q + 1) / 2);
        m0 = in % (q + 1) * kTile;
        n0 = (r * q + in / (q + 1)) * f.bn;
    } else {
        m0 = i % f.tm * kTile;
        n0 = i / f.tm * f.bn;
    }
}

// State that an epilogue warp keeps over the phases.
struct NsEpilogue {
    const NsParams &p;
    const WaitCtl &ctl;
    uint32_t ew, quad, half, lane, tmem_base, leader_tempty;
    int rank, num_pairs;
    uint8_t *slots;
    float *diag;        // 32 values on their way out
    uint64_t *landed, *tfull_bar;
    int acc, pending;   // pending: slots (bits) whose loads have not been waited for
    uint32_t acc_phase, in_phase;
};

// One phase of an epilogue warp; false if the CTA is aborting.
template <int MODE>
__device__ __forceinline__ bool ns_epilogue(NsEpilogue &st, const NsPhase &ph, const CUtensorMap *tm_in0,
                                            const CUtensorMap *tm_in1, const CUtensorMap *tm_out0,
                                            const CUtensorMap *tm_out1) {
    constexpr bool SYM = MODE < kNsUpdate;
    constexpr int kLoads = MODE == kNsGram ? 0 : MODE == kNsPoly ? 1 : 2;   // boxes a chunk reads
    const NsParams &p = st.p;
    const WaitCtl &ctl = st.ctl;
    const uint32_t lane = st.lane, quad = st.quad, half = st.half;
    const int num_tiles = ph.num_tiles, num_pairs = st.num_pairs, first = ph.first;
    const int rows = p.lo, cols = ph.cols;
    uint8_t *const slots = st.slots;
    uint64_t *const landed = st.landed;
    int &acc = st.acc, &pending = st.pending;
    uint32_t &acc_phase = st.acc_phase, &in_phase = st.in_phase;
    const int rank = st.rank;
    const int row_off = rank * 128 + static_cast<int>(quad) * 32, col_off = static_cast<int>(half) * (ph.bn / 2);
    const int chunks = ph.bn / 64;   // of 32 columns, a tile and warp
    // 16-byte unit h of row r of a box (64-byte swizzle)
    auto unit = [](uint8_t *box, int r, int h) {
        return reinterpret_cast<uint4 *>(box + r * 64 + ((h ^ ((r >> 1) & 3)) << 4));
    };
    // chunk c of this pair in this phase (chunk c % chunks of its tile c / chunks): the epilogue's operands, into
    // slot c & 1; nothing past the last
    const int my_chunks = first < num_tiles ? (num_tiles - first + num_pairs - 1) / num_pairs * chunks : 0;
    auto load_chunk = [&](int c) {
        if constexpr (kLoads > 0) {
            if (c >= my_chunks) return;
            int b, m0, n0;
            ns_locate(ph, first + c / chunks * num_pairs, b, m0, n0);
            uint8_t *box = slots + (c & 1) * kSlotBytes;
            const int x = n0 + col_off + 32 * (c % chunks), y = m0 + row_off;
            mbar_arrive_expect_tx(&landed[c & 1], kLoads * kBoxBytes);
            tma_load_3d(box, tm_in0, &landed[c & 1], x, y, b);
            if constexpr (kLoads > 1) tma_load_3d(box + kBoxBytes, tm_in1, &landed[c & 1], x, y, b);
        }
    };
    if (kLoads > 0) {
        if (lane == 0) {
            load_chunk(0);
            load_chunk(1);
        }
        pending = my_chunks >= 2 ? 3 : my_chunks;
    }
    int c = 0;
    for (int t = first; t < num_tiles; t += num_pairs) {
        int b, m0, n0;
        ns_locate(ph, t, b, m0, n0);
        const int row0 = m0 + row_off, row = row0 + static_cast<int>(lane);
        const bool mirror = SYM && n0 >= m0 + kTile;   // (beside the diagonal's block of rows)
        // the row's entry of A's or B's diagonal, and (polynomial) a column's of each chunk by lane
        float diag = 0.f, dcol[4];
        if (MODE != kNsGram && row < rows)
            diag = __ldcg((MODE == kNsPoly ? p.da : p.db) + static_cast<int64_t>(b) * p.ldd + row);
        if constexpr (MODE == kNsPoly) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int cc = n0 + col_off + 32 * j + static_cast<int>(lane);
                dcol[j] = j < chunks && cc < cols ? __ldcg(p.da + static_cast<int64_t>(b) * p.ldd + cc) : 0.f;
            }
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&st.tfull_bar[acc], acc_phase, ctl, DG_DEV_TIMEOUT))) return false;
        tc_fence_after_sync();
#pragma unroll 1
        for (int j = 0; j < chunks; ++j, ++c) {
            const int s = c & 1, col = n0 + col_off + 32 * j;
            uint8_t *box0 = slots + s * kSlotBytes, *box1 = box0 + kBoxBytes;
            uint32_t v[2][16];
            const uint32_t at = st.tmem_base + ((quad * 32) << 16) + acc * kTile + col_off + 32 * j;
            tmem_ld_32x32b_x16(at, v[0]);
            tmem_ld_32x32b_x16(at + 16, v[1]);
            if constexpr (kLoads > 0) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&landed[s], (in_phase >> s) & 1u, ctl, DG_DEV_TIMEOUT)))
                    return false;
                in_phase ^= 1u << s;
                pending &= ~(1 << s);
            }
            tmem_ld_wait();
            reg_fence16(v[0]);
            reg_fence16(v[1]);
            if (j == chunks - 1) {   // the accumulator has been read
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(st.leader_tempty + acc * 8);
            }
            if constexpr (MODE == kNsPoly) {
                if (j > 0) {   // (this chunk's columns in the first place)
                    dcol[0] = dcol[1];
                    dcol[1] = dcol[2];
                    dcol[2] = dcol[3];
                }
            }
            const bool in = row0 < rows && col < cols;   // (else nothing of the chunk is stored)
            if constexpr (kLoads == 0) {
                // the slot's stores have read it (the other slot's may still run)
                if (lane == 0) bulk_wait_group_read<1>();
                __syncwarp();
            }
            float on_diag = 0.f;
            // 8 columns at a time, in place: f in units of 2^-12
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint32_t *x = v[h >> 1] + 8 * (h & 1);
                float f[8];
                uint32_t w0[4], w1[4];
                if constexpr (kLoads > 0) {
                    const uint4 q = *unit(box0, lane, h);
                    w0[0] = q.x; w0[1] = q.y; w0[2] = q.z; w0[3] = q.w;
                }
                if constexpr (kLoads > 1) {
                    const uint4 q = *unit(box1, lane, h);
                    w1[0] = q.x; w1[1] = q.y; w1[2] = q.z; w1[3] = q.w;
                }
                if constexpr (MODE == kNsGram) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(x[i]) * (1.0f / kScale);
                } else if constexpr (MODE == kNsPoly) {
                    float dc[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) dc[i] = __shfl_sync(0xFFFFFFFFu, dcol[0], 8 * h + i);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 r = half2_values(w0[i]);
                        f[2 * i] = fmaf(fmaf(p.cc, diag + dc[2 * i], p.cb), r.x,
                                        p.cc * (1.0f / kScale) * __uint_as_float(x[2 * i]));
                        f[2 * i + 1] = fmaf(fmaf(p.cc, diag + dc[2 * i + 1], p.cb), r.y,
                                            p.cc * (1.0f / kScale) * __uint_as_float(x[2 * i + 1]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 hi = half2_values(w0[i]), lo = half2_values(w1[i]);
                        f[2 * i] = fmaf(p.ca + diag, hi.x + lo.x, (1.0f / kScale) * __uint_as_float(x[2 * i]));
                        f[2 * i + 1] = fmaf(p.ca + diag, hi.y + lo.y, (1.0f / kScale) * __uint_as_float(x[2 * i + 1]));
                    }
                }
                if constexpr (SYM) {
                    // the diagonal goes out in FP32: the chunk whose columns are the warp's rows has all
                    // of the warp's, one a lane (taken by selects: branches cost a microsecond here)
                    const int on = col == row0 ? static_cast<int>(lane) - 8 * h : -1;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        on_diag = i == on ? f[i] : on_diag;
                        f[i] = i == on ? 0.f : f[i];
                    }
                }
                if constexpr (MODE == kNsLast) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= 1.0f / kScale;
                    if (!p.out_tma) {
                        // rows that TMA cannot address: element by element
                        uint16_t *out = p.out + b * p.out_batch;
                        const bool tall = p.rows > p.cols;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int cc = col + 8 * h + i;
                            if (row >= rows || cc >= cols) continue;
                            const __nv_bfloat16 o = __float2bfloat16_rn(f[i]);
                            out[tall ? static_cast<int64_t>(cc) * p.ldo + row : static_cast<int64_t>(row) * p.ldo + cc] =
                                *reinterpret_cast<const uint16_t *>(&o);
                        }
                    } else if (p.rows > p.cols) {
                        // (box1: every lane has read its own unit h of the low plane, the others not;
                        // the transposed box is written once all have, below)
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[h >> 1][8 * (h & 1) + i] = __float_as_uint(f[i]);
                    } else {
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                            o[i] = *reinterpret_cast<const uint32_t *>(&b2);
                        }
                        *unit(box0, lane, h) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                } else if constexpr (MODE == kNsUpdate) {
                    uint32_t o[4], l[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) split2(f[2 * i], f[2 * i + 1], o[i], l[i]);
                    *unit(box0, lane, h) = make_uint4(o[0], o[1], o[2], o[3]);
                    *unit(box1, lane, h) = make_uint4(l[0], l[1], l[2], l[3]);
                } else {
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = half2_bits(f[2 * i], f[2 * i + 1]);
                    *unit(box0, lane, h) = make_uint4(o[0], o[1], o[2], o[3]);
                    if (mirror) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint16_t e = static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1)));
                            uint8_t *const at_unit = reinterpret_cast<uint8_t *>(unit(box1, 8 * h + i, lane >> 3));
                            *reinterpret_cast<uint16_t *>(at_unit + 2 * (lane & 7)) = e;
                        }
                    }
                }
            }
            if constexpr (SYM) {
                on_diag *= 1.0f / kScale;   // (as it is, not scaled)
                if (col == row0) {
                    // (the copy of the diagonal chunk before, which may be the chunk before, has read it)
                    if (lane == 0) bulk_wait_group_read<0>();
                    __syncwarp();
                    st.diag[lane] = MODE == kNsGram ? on_diag : fmaf(diag, fmaf(p.cc, diag, p.cb), on_diag);
                }
            }
            if constexpr (MODE == kNsLast) {
                if (p.out_tma && p.rows > p.cols) {
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const __nv_bfloat16 o = __float2bfloat16_rn(__uint_as_float(v[e >> 4][e & 15]));
                        uint8_t *const at_unit = reinterpret_cast<uint8_t *>(unit(box0, e, lane >> 3));
                        *reinterpret_cast<__nv_bfloat16 *>(at_unit + 2 * (lane & 7)) = o;
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (in && (MODE != kNsLast || p.out_tma)) {
                    if (MODE == kNsLast && p.rows > p.cols) {
                        tma_store_3d(tm_out0, box0, row0, col, b);
                    } else {
                        tma_store_3d(tm_out0, box0, col, row0, b);
                        if (MODE == kNsUpdate) tma_store_3d(tm_out1, box1, col, row0, b);
                        if (mirror) tma_store_3d(tm_out0, box1, row0, col, b);
                        if (SYM && col == row0)   // (rows past lo are padding there)
                            bulk_store((MODE == kNsGram ? p.da : p.db) + static_cast<int64_t>(b) * p.ldd + row0, st.diag, 128);
                    }
                }
                bulk_commit_group();
                // two chunks on: of this tile, or of this pair's next (a phase ends with a wait for all stores)
                if (kLoads > 0 && c + 2 < my_chunks) {
                    bulk_wait_group_read<0>();
                    load_chunk(c + 2);
                }
            }
            if (kLoads > 0 && c + 2 < my_chunks) pending |= 1 << s;
            __syncwarp();
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    // the phase's results are in memory before its arrival
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
    return true;
}

// Waits until a group's counter (the low half of its word) has come to `target`; false if it does not
// within the limit or some CTA has given up (the high half).
__device__ __noinline__ bool ns_grid_wait(const uint64_t *counter, uint32_t target, const WaitCtl &ctl) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i) {
            uint64_t w;
            asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(counter) : "memory");
            if (static_cast<int32_t>(static_cast<uint32_t>(w) - target) >= 0) return true;
            if ((w >> 32) != 0 || *ctl.abort) {
                *ctl.abort = 1;
                return false;
            }
        }
        if (global_timer_ns() - t0 > ctl.timeout_ns) {
            if (ctl.status) atomicOr(ctl.status, DG_DEV_TIMEOUT);
            *ctl.abort = 1;
            return false;
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    dg_ns_products_kernel(const __grid_constant__ NsMaps maps, const __grid_constant__ NsParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int stage_bytes = ring_stage_bytes(p.bn_sym, p.bn_update), stages = ring_stages(p.bn_sym, p.bn_update);
    uint8_t *smem_epi = smem + kRingBytes;
    float *diag_out = reinterpret_cast<float *>(smem_epi + kEpiBytes);   // 32 an epilogue warp
    uint64_t *bars = reinterpret_cast<uint64_t *>(diag_out + 32 * kEpiWarps);
    uint64_t *full_bar = bars;                   // [stages] leader: both CTAs' stages landed
    uint64_t *empty_bar = full_bar + kMaxStages; // [stages] both: MMAs done with the stage
    uint64_t *tfull_bar = empty_bar + kMaxStages;   // [2] both: accumulator complete
    uint64_t *tempty_bar = tfull_bar + 2;        // [2] leader: both epilogues drained
    uint64_t *drain_bar = tempty_bar + 2;
    uint64_t *phase_bar = drain_bar + 1;         // [2] the grid has finished the group's phase before
    uint64_t *in_bar = phase_bar + 2;            // [kEpiWarps][2] an epilogue warp's boxes landed
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(in_bar + 2 * kEpiWarps);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    uint32_t *done = tmem_holder + 2;            // [2] epilogue warps that have finished a group's phases

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;
    const int pair_id = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const int phases = 3 * p.steps, groups = p.group0 < p.batch ? 2 : 1, turns = phases + groups - 1;

    if (warp == 0) {
        for (uint64_t *b = bars + lane; b < in_bar + 2 * kEpiWarps; b += 32)
            mbar_init(b, b >= tempty_bar && b < tempty_bar + 2 ? 2 * kEpiWarps : 1);
        if (lane == 0) {
            *abort_flag = 0;
            done[0] = done[1] = 0u;
        }
        fence_mbar_init();
        if (lane == 0) {
            const CUtensorMap *m = reinterpret_cast<const CUtensorMap *>(&maps);
            for (unsigned i = 0; i < sizeof(maps) / sizeof(CUtensorMap); ++i) tma_prefetch_desc(m + i);
        }
    }
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

    if (warp == 0) {
        const uint32_t leader_full = mapa_shared(smem_u32(full_bar), 0);
        int slot = 0;
        uint32_t phase = 0, issued = 0;
        bool drop = (p.debug_flags & DG_DEBUG_DROP_ONE_LOAD) && pair_id == 0;
        for (int turn = 0; turn < turns; ++turn)
        for (int g = 0; g < groups; ++g) {
            const int i = turn - g;
            const NsPhase f = ns_phase(p, turn, g, pair_id, num_pairs);
            if (f.first >= f.num_tiles) continue;   // (nothing to do: nothing to wait for)
            if (i > 0) {
                bool ok = true;
                if (lane == 0) {
                    ok = ns_grid_wait(p.sync + g, ns_finished(p, i, g), ctl);
                    // the other CTAs' results, written by TMA and plain stores, are read by TMA
                    asm volatile("fence.proxy.async.global;" ::: "memory");
                    if (ok) mbar_arrive(phase_bar + g);
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) goto prod_done;
            }
            const CUtensorMap *ta = f.mode == kNsGram ? &maps.xk[f.step & 1] : f.mode == kNsPoly ? &maps.a : &maps.b;
            const CUtensorMap *tb = f.mode == kNsGram   ? &maps.xkb[f.step & 1]
                                    : f.mode == kNsPoly ? &maps.ab
                                                        : &maps.xn[f.step & 1];
            const bool b_mn = f.mode >= kNsUpdate;
            const int plane = b_mn ? ns_kblocks(kNsPoly, p.lo, p.hi) : f.nkb;   // K-blocks of X's high plane
            // this CTA's half of the columns: bn / 2 rows of 64 K, or boxes of 64 columns (one swizzle
            // atom, of which the MMA reads bn / 2 where that is less) x 64 K rows
            const uint32_t stage = 16384u + (b_mn ? (f.bn == kTile ? 16384u : 8192u) : static_cast<uint32_t>(f.bn) * 64u);
            for (int t = f.first; t < f.num_tiles; t += num_pairs) {
                int b, m0, n0;
                ns_locate(f, t, b, m0, n0);
                for (int kb = 0; kb < f.nkb; ++kb) {
                    if (!mbar_wait_warp(&empty_bar[slot], phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto prod_done;
                    if (drop) {
                        drop = false;   // diagnostic: leave this stage empty
                    } else {
                        if (elect_one()) {
                            const uint32_t fb = leader_full + slot * 8;
                            uint8_t *sa = smem + slot * stage_bytes, *sb = sa + 16384;
                            const int n = n0 + rank * (f.bn / 2), k = (kb < plane ? kb : kb - plane) * kKBlock;
                            if (leader) mbar_arrive_expect_tx(&full_bar[slot], 2 * stage);
                            tma_load_3d_pair(sa, ta, fb, k, m0 + rank * 128, b);
                            if (b_mn) {
                                const CUtensorMap *tp = kb < plane ? tb : &maps.xln;
                                tma_load_3d_pair(sb, tp, fb, n, k, b);
                                if (f.bn == kTile) tma_load_3d_pair(sb + 8192, tp, fb, n + 64, k, b);
                            } else {
                                tma_load_3d_pair(sb, tb, fb, k, n, b);
                            }
                        }
                        __syncwarp();
                        issued |= 1u << slot;
                    }
                    if (++slot == stages) { slot = 0; phase ^= 1; }
                }
            }
        }
    prod_done:
        if (lane == 0 && leader)
            for (int s = 0; s < stages; ++s)
                if (issued & (1u << s)) mbar_wait_drain(&full_bar[s], s < slot ? phase : phase ^ 1, ctl);
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            int slot = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            const uint64_t a0 = make_desc_kmajor_sw128(smem_u32(smem));
            for (int turn = 0; turn < turns; ++turn)
            for (int g = 0; g < groups; ++g) {
                const NsPhase f = ns_phase(p, turn, g, pair_id, num_pairs);
                const bool b_mn = f.mode >= kNsUpdate;
                // FP16 x FP16 -> FP32, M = 256, N = bn (bit 16: B MN-major)
                const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(f.bn >> 3) << 17) | ((kTile >> 4) << 24) |
                                       (b_mn ? 1u << 16 : 0u);
                // (MN-major: the two 64-column atoms 8192 bytes apart, 8 K rows 1024)
                const uint64_t b0 = b_mn ? make_smem_desc(smem_u32(smem) + 16384, 8192, 1024, kSwizzle128B)
                                         : make_desc_kmajor_sw128(smem_u32(smem) + 16384);
                const uint64_t step_b = b_mn ? (2048 >> 4) : 2;   // 16 K: 16 rows, or 32 bytes along a row
                for (int t = f.first; t < f.num_tiles; t += num_pairs) {
                    if (!mbar_wait_cluster_warp(&tempty_bar[acc], acc_phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto mma_done;
                    tc_fence_after_sync();
                    const uint32_t d = tmem_base + acc * kTile;
                    for (int kb = 0; kb < f.nkb; ++kb) {
                        // (a tile's first stage may follow phases that have no tile for this pair: the
                        // limit is far above a phase)
                        if (!mbar_wait_warp(&full_bar[slot], phase, ctl, DG_DEV_TIMEOUT)) goto mma_done;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint64_t a = a0 + slot * (stage_bytes >> 4), b = b0 + slot * (stage_bytes >> 4);
#pragma unroll
                            for (int s = 0; s < 4; ++s) mma_f16_pair(d, a + 2 * s, b + step_b * s, idesc, (kb | s) != 0);
                            tc_commit_pair(&empty_bar[slot], 0x3);
                        }
                        __syncwarp();
                        if (++slot == stages) { slot = 0; phase ^= 1; }
                    }
                    if (elect_one()) tc_commit_pair(&tfull_bar[acc], 0x3);
                    __syncwarp();
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                }
            }
        mma_done:
            if (elect_one()) {
                tc_commit_pair(drain_bar, 0x1);
                mbar_wait(drain_bar, 0, ctl, DG_DEV_TIMEOUT);
            }
            __syncwarp();
        }
    } else {
        const uint32_t ew = warp - 2;
        NsEpilogue st{p, ctl, ew, warp & 3, ew >> 2, lane, tmem_base, mapa_shared(smem_u32(tempty_bar), 0), rank, num_pairs,
                      smem_epi + ew * 2 * kSlotBytes, diag_out + 32 * ew, in_bar + 2 * ew, tfull_bar, 0, 0, 0u, 0u};
        bool ok = true;
        uint32_t waited = 0;   // parities of phase_bar
        for (int turn = 0; turn < turns && ok; ++turn)
        for (int g = 0; g < groups && ok; ++g) {
            const int i = turn - g;
            const NsPhase f = ns_phase(p, turn, g, pair_id, num_pairs);
            if (f.first >= f.num_tiles) continue;
            if (i > 0) {
                ok = mbar_wait_warp(phase_bar + g, (waited >> g) & 1u, ctl, DG_DEV_TIMEOUT);
                waited ^= 1u << g;
                if (!ok) break;
                asm volatile("fence.proxy.async.global;" ::: "memory");   // (as the producer's)
            }
            const CUtensorMap *xh = &maps.xh[f.step & 1], *next = &maps.xh[(f.step & 1) ^ 1];
            if (f.mode == kNsGram) ok = ns_epilogue<kNsGram>(st, f, nullptr, nullptr, &maps.ea, nullptr);
            else if (f.mode == kNsPoly) ok = ns_epilogue<kNsPoly>(st, f, &maps.ea, nullptr, &maps.eb, nullptr);
            else if (f.mode == kNsUpdate) ok = ns_epilogue<kNsUpdate>(st, f, xh, &maps.xl, next, &maps.xl);
            else ok = ns_epilogue<kNsLast>(st, f, xh, &maps.xl, &maps.out, nullptr);
            if (!ok) break;
            // The CTA's last warp to finish the phase counts its tiles.  A warp's results (its boxes,
            // complete since the wait for them) are released to the CTA by its count, and by the last
            // warp's, which has acquired the others', to the grid: one release at the grid's scope
            // (one a warp and no count in the CTA: 0.15 to 0.4 us more a phase).
            __syncwarp();
            if (lane == 0 && i + 1 < phases) {
                uint32_t before;
                asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;"
                             : "=r"(before)
                             : "r"(smem_u32(done + g))
                             : "memory");
                if (before % kEpiWarps == kEpiWarps - 1)
                    asm volatile("red.release.gpu.global.add.u64 [%0], %1;" ::"l"(p.sync + g),
                                 "l"(static_cast<uint64_t>((f.num_tiles - f.first + num_pairs - 1) / num_pairs))
                                 : "memory");
            }
        }
        // (an aborted loop leaves no load landing in shared memory after the CTA is gone)
        if (lane == 0) {
            for (int s = 0; s < 2; ++s)
                if (st.pending & (1 << s)) mbar_wait_drain(&st.landed[s], (st.in_phase >> s) & 1u, ctl);
            bulk_wait_group<0>();
        }
        __syncwarp();
    }
    // a CTA that gave up tells the others
    if (lane == 0 && *abort_flag)
        for (int g = 0; g < groups; ++g) atomicOr(reinterpret_cast<uint32_t *>(p.sync + g) + 1, 1u);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// 3-D map of planes [batch][rows][ld] of 16-bit values: boxes of 64 elements (128 bytes) x box_rows as
// operands, of 32 x 32 elements for the epilogue.
bool encode_plane(CUtensorMap *map, const uint16_t *base, int64_t cols, int64_t rows, int64_t ld, int64_t batch_stride,
                  int64_t batch, uint32_t box_rows, bool epi = false) {
    TensorMapEncodeFn fn = host_encode();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(batch_stride) * 2};
    const cuuint32_t box[3] = {epi ? 32u : kKBlock, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, epi ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              epi ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Co-resident CTA pairs on the current device, at most num_sms / 2.
int max_pairs(int num_sms) {
    static std::mutex mu;
    static int cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int &v = cache[dev];
    if (v == 0) {
        if (cudaFuncSetAttribute(dg_ns_products_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
            return 0;
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
        if (cudaOccupancyMaxActiveClusters(&v, dg_ns_products_kernel, &cfg) != cudaSuccess) v = 0;
    }
    return v * 2 > num_sms ? num_sms / 2 : v;
}

// Tiles of a matrix's product with tiles of bn columns (as ns_shape counts them).
int64_t count_tiles(const NsParams &p, bool sym, int bn) {
    const int64_t tm = up(p.lo, kTile) / kTile, tn = up(sym ? p.lo : p.hi, bn) / bn, r = kTile / bn, q = tn / r;
    return sym ? r * (q * (q + 1) / 2) + (tn - r * q) * (q + 1) : tm * tn;
}

// Columns of a product's tiles: 256, or where those are few, 128 or 64.  A tile's time is modelled as its
// K-blocks times the cycles of one (the operands' loads set them: 16 KB of rows and 64 bytes
// a column at about 55 bytes a cycle) and its epilogue (a chunk of 32 columns after another,
// about 1500 cycles each), which only the last tile of a pair does not hide.  Measured, chosen against 256
// throughout: 250x1000 127 us and 168, 1024x1024 149 and 217.
int choose_bn(const NsParams &p, bool sym, int pairs) {
    int best = 256;
    double least = 0.0;
    for (int bn : {256, 128, 64}) {
        const int64_t n = count_tiles(p, sym, bn) * p.batch;
        // (symmetric: the mean of the products along the long side and the short)
        const int64_t nkb = sym ? (up(p.hi, kKBlock) + up(p.lo, kKBlock)) / kKBlock / 2 + 1 : ns_kblocks(kNsUpdate, p.lo, p.hi);
        const double t = static_cast<double>((n + pairs - 1) / pairs) * nkb * (16384 + 64 * bn) / 55.0 +
                         1500.0 * (bn / 64);
        if (bn == 256 || t < 0.95 * least) {
            best = bn;
            least = t;
        }
    }
    return best;
}

// Modelled time in us of `steps` steps with tiles of these columns, in one group or in two: each pair's
// tiles one after another in turn order (ns_phase), the phase's no sooner than 3.3 us (the chain of counter,
// load, epilogue and store, of which a tile's columns past 64 add their epilogue) after the
// last tile of the group's phase before.  Tiles cost as in choose_bn, at 1.9 GHz.  The second group's waits and
// its tiles' loads beside the first's: 1.2 us a phase.
double model_time(const NsParams &p, int steps, int bn_sym, int bn_update, int groups, int pairs) {
    constexpr int kMax = 128;
    if (pairs > kMax) pairs = kMax;
    float busy[kMax] = {}, done[2] = {};
    float cost[3], tail[3];
    int64_t tiles[3];
    for (int m = 0; m < 3; ++m) {
        const int bn = m < kNsUpdate ? bn_sym : bn_update;
        const int64_t nkb = ns_kblocks(m, p.lo, p.hi);
        const float epilogue = 0.79f * (bn / 64), loads = nkb * (16384 + 64 * bn) / 104500.0f;
        cost[m] = loads > epilogue ? loads : epilogue;
        tail[m] = 3.3f + epilogue - 0.79f;
        tiles[m] = count_tiles(p, m < kNsUpdate, bn);
    }
    const int phases = 3 * (steps < 3 ? steps : 3);
    for (int turn = 0; turn < phases + groups - 1; ++turn) {
        int first = 0;
        for (int g = 0; g < groups; ++g) {
            const int i = turn - g;
            if (i < 0 || i >= phases) continue;
            const int64_t n = tiles[i % 3] * (groups == 1 ? p.batch : g == 0 ? p.batch - p.batch / 2 : p.batch / 2);
            const int64_t each = n / pairs;
            const int more = static_cast<int>(n % pairs);   // pairs from `first` on that have one more
            float end = done[g];
            for (int q = 0; q < pairs; ++q) {
                const int at = q >= first ? q - first : q - first + pairs;
                const int64_t mine = each + (at < more ? 1 : 0);
                if (mine == 0) continue;
                const float t = (busy[q] > done[g] ? busy[q] : done[g]) + mine * cost[i % 3];
                busy[q] = t;
                end = t > end ? t : end;
            }
            done[g] = end + tail[i % 3];
            if (g == 0) first = more;
        }
    }
    return (done[0] > done[1] ? done[0] : done[1]) + (groups > 1 ? 1.2 * phases : 0.0);
}

// Columns of the products' tiles and the matrices of the first group.  Two groups let one have tiles
// while the other waits for its phase's last, and let a symmetric product's few tiles run beside an
// update's many; they cost where a phase alone fills the pairs.  The model decides, between tiles of 256 and 128
// columns (64, two groups against one: 8x512x512 125 us and 115, 700x40x64 305 and 294).  Measured, two
// against one: 2x2112x1536 286 us and 300, 4x1024x1024 196 and 207, 8x1024x1024 293 and 319, 4x2048x2048
// 533 and 583, 16x512x1024 213 and 224, 3x2048x7168 1165 and 1252, 4x2048x7168 1414 and 1463; left as one
// group: 2x1536x1536 246 and 244, 2x1024x4096 310 and 257, 3x1408x2048 367 and 320, 2x2048x7168 822 and 777.
void choose_tiles(NsParams &p, int steps, int pairs) {
    p.bn_sym = choose_bn(p, true, pairs);
    p.bn_update = choose_bn(p, false, pairs);
    p.group0 = p.batch;
    if (p.batch < 2) return;
    double least = model_time(p, steps, p.bn_sym, p.bn_update, 1, pairs);
    for (int s : {256, 128})
        for (int u : {256, 128}) {
            const double t = model_time(p, steps, s, u, 2, pairs);
            if (t < least) {
                least = t;
                p.bn_sym = s;
                p.bn_update = u;
                p.group0 = p.batch - p.batch / 2;
            }
        }
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

// Two high planes, the low plane, A and B, their diagonals, the norm's partial sums, the grid's counter;
// rows of whole 64-element (128-byte) lines.
int64_t ns_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    const int64_t lo = rows < cols ? rows : cols, hi = rows < cols ? cols : rows;
    return batch * (2 * lo * (3 * up(hi, 64) + 2 * up(lo, 64)) + 8 * kMaxPartial + 8 * up(lo, 32)) + 128;
}

cudaError_t launch_newton_schulz(NsParams p, int steps, bool bf16, int num_sms, cudaStream_t stream, NsConfig *config) {
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
    p.sync = reinterpret_cast<uint64_t *>(take(128));
    p.partial = reinterpret_cast<double *>(take(8ll * kMaxPartial * p.batch));
    p.ldd = up(p.lo, 32);
    p.da = reinterpret_cast<float *>(take(4 * p.ldd * p.batch));
    p.db = reinterpret_cast<float *>(w);
    p.dense = p.ldg == p.cols;
    const int64_t segs = p.dense ? (static_cast<int64_t>(p.rows) * p.cols + 8191) / 8192
                                 : p.rows * ((p.cols + 8191ll) / 8192);
    // (by the matrix alone, as its sum's order)
    p.num_partial = static_cast<int>(segs < kMaxPartial ? segs : kMaxPartial);
    cudaError_t e = launch_simple(bf16 ? dg_ns_norm_kernel<true> : dg_ns_norm_kernel<false>,
                                  dim3(p.num_partial, p.batch), p, stream);
    if (e != cudaSuccess) return e;
    const bool tall = p.rows > p.cols;
    if (tall)
        e = launch_simple(bf16 ? dg_ns_split_kernel<true, true> : dg_ns_split_kernel<false, true>,
                          dim3((p.cols + 63) / 64, (p.rows + 255) / 256, p.batch), p, stream);
    else
        e = launch_simple(bf16 ? dg_ns_split_kernel<true, false> : dg_ns_split_kernel<false, false>,
                          dim3((p.cols + 2047) / 2048, (p.rows + 7) / 8, p.batch), p, stream);
    if (e != cudaSuccess) return e;
    // operands: X along K (Gram), X as [K][N], A and B; epilogue boxes of the planes, A, B and the output
    const int pairs = max_pairs(num_sms);
    if (pairs <= 0) return cudaErrorInvalidConfiguration;
    choose_tiles(p, steps, pairs);
    // (no more pairs than the phase that has most tiles)
    const int64_t tiles_sym = count_tiles(p, true, p.bn_sym) * p.batch;
    int64_t tiles = count_tiles(p, false, p.bn_update) * p.batch;
    if (tiles_sym > tiles) tiles = tiles_sym;
    NsMaps maps;
    const int64_t px = p.lo * p.ldx, pa = p.lo * p.lda;
    bool ok = true;
    for (int i = 0; i < 2; ++i)
        ok &= encode_plane(&maps.xk[i], p.xh[i], p.hi, p.lo, p.ldx, px, p.batch, 128) &&
              encode_plane(&maps.xn[i], p.xh[i], p.hi, p.lo, p.ldx, px, p.batch, kKBlock) &&
              encode_plane(&maps.xkb[i], p.xh[i], p.hi, p.lo, p.ldx, px, p.batch, p.bn_sym / 2) &&
              encode_plane(&maps.xh[i], p.xh[i], p.hi, p.lo, p.ldx, px, p.batch, 32, true);
    ok &= encode_plane(&maps.xl, p.xl, p.hi, p.lo, p.ldx, px, p.batch, 32, true) &&
          encode_plane(&maps.xln, p.xl, p.hi, p.lo, p.ldx, px, p.batch, kKBlock) &&
          encode_plane(&maps.a, p.a, p.lo, p.lo, p.lda, pa, p.batch, 128) &&
          encode_plane(&maps.ab, p.a, p.lo, p.lo, p.lda, pa, p.batch, p.bn_sym / 2) &&
          encode_plane(&maps.b, p.b, p.lo, p.lo, p.lda, pa, p.batch, 128) &&
          encode_plane(&maps.ea, p.a, p.lo, p.lo, p.lda, pa, p.batch, 32, true) &&
          encode_plane(&maps.eb, p.b, p.lo, p.lo, p.lda, pa, p.batch, 32, true);
    if (!ok) return cudaErrorInvalidValue;
    // the output by TMA where its rows (and matrices) start on 16 bytes
    p.out_tma = (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0 && p.ldo % 8 == 0 &&
                (p.batch == 1 || p.out_batch % 8 == 0) &&
                encode_plane(&maps.out, p.out, p.cols, p.rows, p.ldo, p.batch == 1 ? p.ldo * p.rows : p.out_batch,
                             p.batch, 32, true);
    if (!p.out_tma) maps.out = maps.ea;   // not used
    p.steps = steps;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // the CTAs wait for one another
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3(2 * static_cast<int>(tiles < pairs ? tiles : pairs));
    *config = {p.bn_sym, p.bn_update, ring_stages(p.bn_sym, p.bn_update), static_cast<int>(cfg.gridDim.x), 3, p.group0};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dg_ns_products_kernel, maps, p);
}

}  // namespace dg
