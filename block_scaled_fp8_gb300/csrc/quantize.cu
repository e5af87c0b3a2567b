// FP8 quantiser: bf16 or FP32 values -> E4M3 codes and packed UE8M0 scales, with a scale for
// each 1x128 of a row (the products along the columns), each 128x1 of a column (the products along
// the rows: weight gradients), both in one read, or each 128x128 block (weights).  The scale
// rule is in quant.cuh.
//
// Memory bound: 2 or 4 bytes read and 1 or 2 written a value, a few operations each.  A CTA takes a
// tile of 128 rows x 128 columns and keeps it in registers: 16 lanes hold a row's 128 values, 8 each,
// so a row's amax is 4 shuffles, and a thread's rows are 16 apart, so a column's amax is a maximum
// over the thread's own rows, one shuffle, and one pass through shared memory.  Each value is read
// once whatever is written.  For rows alone a tile is 16 rows x 128 or 512 columns.
// Measured, bf16 8192x7168 both ways: 36.6 us, 6.4 TB/s of the 236 MB, with 57 % of the issue slots in
// use (49 us with twice the instructions, before maxima and products went two values at a time);
// blocks of 8 FP32 matrices 4096x7168: 165 us, 7.1 TB/s; rows of 96x7168: 5.2 us, a launch.
#include <cuda_bf16.h>

#include "dg_internal.h"
#include "quant.cuh"

namespace dg {
namespace {

constexpr int kQThreads = 256;
constexpr uint32_t kInf = 0x7F800000u;

// 8 consecutive values of a row as they lie: 4 words of bf16 pairs, or 8 FP32 words
template <bool BF16>
constexpr int kWords = BF16 ? 4 : 8;

// The values of a row from col on; zero past the columns (FULL: there are none past them)
template <bool BF16, bool FULL>
__device__ __forceinline__ void load8(const QuantParams &p, const char *at, int col, uint32_t (&w)[kWords<BF16>]) {
    if (FULL || col + 8 <= p.cols) {
        const uint4 *q = reinterpret_cast<const uint4 *>(at);
#pragma unroll
        for (int i = 0; i < kWords<BF16> / 4; ++i) {
            const uint4 x = __ldcg(q + i);   // (read once, so past L1)
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kWords<BF16>; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < p.cols) {
                if constexpr (BF16)
                    w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(at)[i]) << (16 * (i & 1));
                else
                    w[i] = reinterpret_cast<const uint32_t *>(at)[i];
            }
    }
}

// The larger magnitude of two words, element by element, with some sign (one instruction; masked
// where it is used).  A NaN never wins; an infinity does.
template <bool BF16>
__device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF16) asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.xorsign.abs.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A word's larger magnitude as FP32 bits (a NaN only where all of it is)
template <bool BF16>
__device__ __forceinline__ uint32_t magnitude(uint32_t m) {
    if constexpr (BF16) return (amax2<true>(m, __byte_perm(m, m, 0x1032)) & 0x7FFFu) << 16;
    else return m & 0x7FFFFFFFu;
}

// Infinities become NaN, so that they do not count and get the NaN code.
template <bool BF16, int N>
__device__ __forceinline__ void drop_infinities(uint32_t (&v)[N][kWords<BF16>]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < kWords<BF16>; ++j) {
            const uint32_t w = v[i][j];
            if constexpr (BF16) {
                if ((w & 0x7FFF0000u) == kInf) v[i][j] = (v[i][j] & 0xFFFFu) | 0x7FC00000u;
                if ((w & 0x7FFFu) == 0x7F80u) v[i][j] = (v[i][j] & 0xFFFF0000u) | 0x7FC0u;
            } else {
                if ((w & 0x7FFFFFFFu) == kInf) v[i][j] = 0x7FC00000u;
            }
        }
}

// 1 / scale of a byte as a factor of the words' elements: FP32, or bf16 twice (a power of two in
// bf16's range: products are exact, or so small that their code is 0)
template <bool BF16>
__device__ __forceinline__ uint32_t factor(uint32_t byte) {
    return BF16 ? (254u - byte) * 0x00800080u : (254u - byte) << 23;
}

// Codes of the 8 values over their scales: word j (or value j) times factor f(j)
template <bool BF16, bool FULL, typename F>
__device__ __forceinline__ void put_codes(const QuantParams &p, uint8_t *at, int col, const uint32_t (&w)[kWords<BF16>],
                                          F f) {
    float v[8];
#pragma unroll
    for (int j = 0; j < kWords<BF16>; ++j) {
        if constexpr (BF16) {
            uint32_t x;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[j]), "r"(f(j)));
            v[2 * j] = __uint_as_float(x << 16);
            v[2 * j + 1] = __uint_as_float(x & 0xFFFF0000u);
        } else {
            v[j] = __uint_as_float(w[j]) * __uint_as_float(f(j));
        }
    }
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        asm("{\n\t.reg .b16 a, b;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
            "mov.b32 %0, {a, b};\n\t}"
            : "=r"(o[j])
            : "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3]));
    if (FULL || col + 8 <= p.cols) {
        *reinterpret_cast<uint2 *>(at) = make_uint2(o[0], o[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < p.cols) at[i] = static_cast<uint8_t>(o[i / 4] >> (8 * (i & 3)));
    }
}

// Row j of the packed words that 128-row block `block` belongs to, its byte, and whether it is the
// last block of its group (whose thread clears the word's unused bytes).
__device__ __forceinline__ void packed_row(const QuantParams &p, const KGroupRows &t, int block, int &word, int &byte,
                                           bool &last) {
    int first = 0, end = (p.rows + 127) / 128, w0 = 0;
    if (t.num_groups > 0) {
        int lo = 0, hi = t.num_groups;   // the group with srow[lo] <= block < srow[lo + 1]
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (t.srow[mid] <= block) lo = mid; else hi = mid - 1;
        }
        first = t.srow[lo];
        end = t.srow[lo + 1];
        w0 = t.prow[lo];
    }
    word = w0 + (block - first) / 4;
    byte = (block - first) & 3;
    last = block + 1 == end;
}

__device__ __forceinline__ void put_byte(uint8_t *word, int byte, uint32_t v, bool last) {
    word[byte] = static_cast<uint8_t>(v);
    if (last)
        for (int b = byte + 1; b < 4; ++b) word[b] = 0;
}

// Largest magnitudes of N rows over the 16 lanes that hold a row's 128 values, as FP32 bits, from each
// lane's own.  bf16: two rows to a word.
template <bool BF16, int N>
__device__ __forceinline__ void row_amax(const uint32_t (&m)[N], uint32_t (&out)[N]) {
    if constexpr (BF16 && N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            // both rows' low halves, both rows' high halves
            uint32_t x = amax2<true>(__byte_perm(m[i], m[i + 1], 0x5410), __byte_perm(m[i], m[i + 1], 0x7632));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) x = amax2<true>(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            out[i] = (x & 0x7FFFu) << 16;
            out[i + 1] = x & 0x7FFF0000u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t x = magnitude<BF16>(m[i]);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) x = amax2<false>(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            out[i] = x & 0x7FFFFFFFu;
        }
    }
}

struct QuantShared {
    uint32_t col[8][128];    // a warp's column amax (bf16: pairs)
    uint32_t inv[128];       // the columns' factors (bf16: pairs)
    uint32_t block[8];
};

// One tile of TR rows x TC columns, 128 x 128 but for rows alone.  MODE: 1 rows, 2 columns, 3 both,
// 4 blocks.  FULL: the tile lies inside the matrix.
template <bool BF16, int MODE, int TR, int TC, bool FULL>
__device__ __forceinline__ void quantize_tile(const QuantParams &p, const KGroupRows &t, QuantShared &s, int ty) {
    constexpr int kLanes = TC / 8, kPass = kQThreads / kLanes;   // threads of a row, rows at a time
    constexpr int N = TR / kPass;       // rows of a thread
    constexpr int W = kWords<BF16>;
    constexpr bool ROWS = MODE == 1 || MODE == 3, COLS = MODE == 2 || MODE == 3;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cl = threadIdx.x % kLanes, rl = threadIdx.x / kLanes;
    const int col0 = blockIdx.x * TC, col = col0 + cl * 8, row0 = ty * TR + rl;
    const int64_t batch = blockIdx.z;
    uint32_t v[N][W];
    {
        constexpr int kSize = BF16 ? 2 : 4;
        const char *x = static_cast<const char *>(p.x) +
                        (batch * p.x_batch + static_cast<int64_t>(row0) * p.ldx + col) * kSize;
        const int64_t step = static_cast<int64_t>(kPass * kSize) * p.ldx;
#pragma unroll
        for (int i = 0; i < N; ++i, x += step) {
            if (FULL || row0 + kPass * i < p.rows) {
                load8<BF16, FULL>(p, x, col, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = 0u;
            }
        }
    }
    // the thread's amax by row or by column, either of which also says whether there is an infinity
    uint32_t rm[N], cm[W], any;
    auto maxima = [&]() {
        any = 0u;
        if constexpr (ROWS) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                rm[i] = v[i][0];
#pragma unroll
                for (int j = 1; j < W; ++j) rm[i] = amax2<BF16>(rm[i], v[i][j]);
                if constexpr (MODE == 1) any = i == 0 ? rm[0] : amax2<BF16>(any, rm[i]);
            }
        }
        if constexpr (MODE != 1) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                cm[j] = v[0][j];
#pragma unroll
                for (int i = 1; i < N; ++i) cm[j] = amax2<BF16>(cm[j], v[i][j]);
                any = j == 0 ? cm[0] : amax2<BF16>(any, cm[j]);
            }
        }
        any = magnitude<BF16>(any);
    };
    maxima();
    if (any == kInf) {
        drop_infinities<BF16, N>(v);
        maxima();
    }
    if constexpr (ROWS) {
        const int gi = blockIdx.x * (TC / 128) + cl / 16;
        const bool last = (gi + 1) * 128 >= p.cols;
        uint32_t amax[N];
        row_amax<BF16, N>(rm, amax);
        uint8_t *q = p.q + static_cast<int64_t>(row0) * p.ldq + col;
        uint8_t *sf = p.sf + (static_cast<int64_t>(gi >> 2) * p.sf_ld + row0) * 4;
        const int64_t step = kPass * p.ldq;
#pragma unroll
        for (int i = 0; i < N; ++i, q += step) {
            const int row = row0 + kPass * i;
            const uint32_t byte = ue8m0_of_amax(amax[i]), f = factor<BF16>(byte);
            if (FULL || row < p.rows) put_codes<BF16, FULL>(p, q, col, v[i], [f](int) { return f; });
            // (rows that pad the words to a multiple of 4: zero)
            if (cl % 16 == 0 && (FULL || (row < p.sf_ld && (TC == 128 || col < p.cols))))
                put_byte(sf + 4 * kPass * i, gi & 3, FULL || row < p.rows ? byte : 0u, last);
        }
    }
    if constexpr (COLS) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            cm[j] = amax2<BF16>(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 16));
            if (lane < 16) s.col[warp][cl * W + j] = cm[j];
        }
        __syncthreads();
        if (threadIdx.x < 16 * W) {
            uint32_t m = s.col[0][threadIdx.x], inv = 0u;
#pragma unroll
            for (int w = 1; w < 8; ++w) m = amax2<BF16>(m, s.col[w][threadIdx.x]);
#pragma unroll
            for (int e = 0; e < (BF16 ? 2 : 1); ++e) {
                const int c = col0 + static_cast<int>(threadIdx.x) * (BF16 ? 2 : 1) + e;
                const uint32_t byte =
                    ue8m0_of_amax(BF16 ? (e ? m & 0x7FFF0000u : (m & 0x7FFFu) << 16) : m & 0x7FFFFFFFu);
                const uint32_t f = factor<BF16>(byte);
                inv = !BF16 ? f : e ? (inv & 0xFFFFu) | (f & 0xFFFF0000u) : f;
                if (c < p.sfk_ld) {
                    int word, at;
                    bool last;
                    packed_row(p, t, ty, word, at, last);
                    put_byte(p.sfk + (static_cast<int64_t>(word) * p.sfk_ld + c) * 4, at, c < p.cols ? byte : 0u, last);
                }
            }
            s.inv[threadIdx.x] = inv;
        }
        __syncthreads();
        uint32_t inv[W];
#pragma unroll
        for (int j = 0; j < W; ++j) inv[j] = s.inv[cl * W + j];
        uint8_t *q = p.qk + static_cast<int64_t>(row0) * p.ldqk + col;
        const int64_t step = kPass * p.ldqk;
#pragma unroll
        for (int i = 0; i < N; ++i, q += step)
            if (FULL || row0 + kPass * i < p.rows)
                put_codes<BF16, FULL>(p, q, col, v[i], [&inv](int j) { return inv[j]; });
        // (the next tile's writes to s.inv come after its own first barrier, and those to s.col after
        // every thread has passed this tile's second)
    }
    if constexpr (MODE == 4) {
        uint32_t m = __reduce_max_sync(0xFFFFFFFFu, any > kInf ? 0u : any);
        if (lane == 0) s.block[warp] = m;
        __syncthreads();
        m = s.block[0];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max(m, s.block[w]);
        const uint32_t byte = ue8m0_of_amax(m), f = factor<BF16>(byte);
        uint8_t *q = p.q + batch * p.q_batch + static_cast<int64_t>(row0) * p.ldq + col;
        const int64_t step = kPass * p.ldq;
#pragma unroll
        for (int i = 0; i < N; ++i, q += step)
            if (FULL || row0 + kPass * i < p.rows) put_codes<BF16, FULL>(p, q, col, v[i], [f](int) { return f; });
        // one byte a row (products along the columns), one a column (along the rows)
        const int i = threadIdx.x & 127;
        if (threadIdx.x < 128) {
            const int gi = blockIdx.x, row = ty * 128 + i;
            if (p.sf != nullptr && row < p.sf_ld)
                put_byte(p.sf + ((batch * ((p.cols + 511) / 512) + (gi >> 2)) * p.sf_ld + row) * 4, gi & 3,
                         row < p.rows ? byte : 0u, col0 + 128 >= p.cols);
        } else {
            const int c = col0 + i;
            if (p.sfk != nullptr && c < p.sfk_ld)
                put_byte(p.sfk + ((batch * ((p.rows + 511) / 512) + (ty >> 2)) * p.sfk_ld + c) * 4, ty & 3,
                         c < p.cols ? byte : 0u, (ty + 1) * 128 >= p.rows);
        }
        __syncthreads();   // s.block is free for the next tile
    }
}

template <bool BF16, int MODE, int TR, int TC = 128>
__global__ void __launch_bounds__(kQThreads, MODE == 1 ? (BF16 ? 6 : 4) : BF16 ? 4 : 2) dg_quantize_kernel(
    const __grid_constant__ QuantParams p, const __grid_constant__ KGroupRows t) {
    static_assert((TR == 128 && TC == 128) || MODE == 1, "columns and blocks have 128 rows and columns");
    __shared__ QuantShared s;
    grid_launch_dependents();
    grid_dependency_wait();
    const int tiles_y = (p.rows + TR - 1) / TR;
    for (int ty = blockIdx.y; ty < tiles_y; ty += gridDim.y) {
        if ((ty + 1) * static_cast<int64_t>(TR) <= p.rows && (blockIdx.x + 1) * static_cast<int64_t>(TC) <= p.cols)
            quantize_tile<BF16, MODE, TR, TC, true>(p, t, s, ty);
        else
            quantize_tile<BF16, MODE, TR, TC, false>(p, t, s, ty);
    }
}

template <bool BF16, int MODE, int TR, int TC = 128>
cudaError_t launch_one(const QuantParams &p, const KGroupRows &t, int batch, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const int ty = (p.rows + TR - 1) / TR;
    cfg.gridDim = dim3((p.cols + TC - 1) / TC, ty < 65535 ? ty : 65535, batch);
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dg_quantize_kernel<BF16, MODE, TR, TC>, p, t);
}

template <bool BF16>
cudaError_t launch_typed(const QuantParams &p, const KGroupRows &t, int batch, int mode, int num_sms,
                         cudaStream_t stream) {
    switch (mode) {
        case 1: {
            // rows alone: a row's scale needs no other row, so tiles have 16.  512 columns keep a
            // warp's loads on few rows and 4 of them a thread in flight (8192x7168 bf16: 24 us against
            // 34 with 128x128); where the matrix is small, 128 columns spread it over four
            // times as many CTAs.
            const int64_t tiles = static_cast<int64_t>((p.cols + 127) / 128) * ((p.rows + 127) / 128);
            if (tiles < 2 * num_sms) return launch_one<BF16, 1, 16>(p, t, batch, stream);
            return launch_one<BF16, 1, 16, 512>(p, t, batch, stream);
        }
        case 2: return launch_one<BF16, 2, 128>(p, t, batch, stream);
        case 3: return launch_one<BF16, 3, 128>(p, t, batch, stream);
        default: return launch_one<BF16, 4, 128>(p, t, batch, stream);
    }
}

}  // namespace

cudaError_t launch_quantize(const QuantParams &p, const KGroupRows &t, int batch, int mode, bool bf16, int num_sms,
                            cudaStream_t stream) {
    return bf16 ? launch_typed<true>(p, t, batch, mode, num_sms, stream)
                : launch_typed<false>(p, t, batch, mode, num_sms, stream);
}

}  // namespace dg
