// FP8 quantiser: bf16 or FP32 values -> E4M3 codes and packed UE8M0 scales, with a scale for
// each 1x128 of a row (the products along the columns), each 128x1 of a column (the products along
// the rows: weight gradients), both in one read, or each 128x128 block (weights).  The scale
// rule is in quant.cuh.
//
// Memory bound: 2 or 4 bytes read and 1 or 2 written a value, a few operations each.  A CTA takes a
// tile of TR rows x 128 columns and keeps it in registers: 16 lanes hold a row's 128 values, 8 each,
// so a row's amax is 4 shuffles, and a thread's rows are 16 apart, so a column's amax is a maximum
// over the thread's own rows, one shuffle, and one pass through shared memory.  Each value is read
// once whatever is written.
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

// The values of a row from col on; zero past the columns
template <bool BF16>
__device__ __forceinline__ void load8(const QuantParams &p, const char *row, int col, uint32_t (&w)[kWords<BF16>]) {
    if (col + 8 <= p.cols) {
        const uint4 *q = reinterpret_cast<const uint4 *>(row + (BF16 ? 2 : 4) * static_cast<int64_t>(col));
#pragma unroll
        for (int i = 0; i < kWords<BF16> / 4; ++i) {
            const uint4 x = __ldcs(q + i);   // (read once)
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kWords<BF16>; ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < p.cols) {
                if constexpr (BF16)
                    w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[col + i]) << (16 * (i & 1));
                else
                    w[i] = reinterpret_cast<const uint32_t *>(row)[col + i];
            }
    }
}

// Value i of the 8
template <bool BF16>
__device__ __forceinline__ float value(const uint32_t (&w)[kWords<BF16>], int i) {
    if constexpr (BF16) return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else return __uint_as_float(w[i]);
}

// max(m, |w|), element by element of a word (m not negative).  A NaN never wins; an infinity does.
template <bool BF16>
__device__ __forceinline__ uint32_t amax_word(uint32_t m, uint32_t w) {
    if constexpr (BF16) {
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&m),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)));
        return *reinterpret_cast<const uint32_t *>(&r);
    } else {
        return __float_as_uint(fmaxf(__uint_as_float(m), fabsf(__uint_as_float(w))));
    }
}

// A word's larger element as FP32 bits
template <bool BF16>
__device__ __forceinline__ uint32_t amax_bits_of(uint32_t m) {
    if constexpr (BF16) return max(m & 0xFFFF0000u, m << 16);
    else return m;
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

__device__ __forceinline__ void store8(const QuantParams &p, uint8_t *row, int col, uint32_t lo, uint32_t hi) {
    if (col + 8 <= p.cols) {
        *reinterpret_cast<uint2 *>(row + col) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < p.cols) row[col + i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

// The 8 values over one scale, or over their columns' scales, to the codes of a row
template <bool BF16>
__device__ __forceinline__ void put_codes(const QuantParams &p, uint8_t *row, int col, const uint32_t (&w)[kWords<BF16>],
                                          const float (&inv)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = cvt_e4m3x2(value<BF16>(w, 2 * j) * inv[2 * j], value<BF16>(w, 2 * j + 1) * inv[2 * j + 1]);
    store8(p, row, col, o[0] | o[1] << 16, o[2] | o[3] << 16);
}
template <bool BF16>
__device__ __forceinline__ void put_codes(const QuantParams &p, uint8_t *row, int col, const uint32_t (&w)[kWords<BF16>],
                                          float inv) {
    const float all[8] = {inv, inv, inv, inv, inv, inv, inv, inv};
    put_codes<BF16>(p, row, col, w, all);
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

// MODE: 1 rows, 2 columns, 3 both, 4 blocks.  TR: rows of a tile (128 but for rows alone).
template <bool BF16, int MODE, int TR>
__global__ void __launch_bounds__(kQThreads, BF16 ? 4 : 2) dg_quantize_kernel(const __grid_constant__ QuantParams p,
                                                                              const __grid_constant__ KGroupRows t) {
    static_assert(TR == 128 || MODE == 1, "columns and blocks have 128 rows");
    constexpr int N = TR / 16;          // rows of a thread
    constexpr int W = kWords<BF16>;
    constexpr bool COLS = MODE == 2 || MODE == 3;
    __shared__ uint32_t s_col[COLS ? 8 : 1][16 * W];   // a warp's column amax
    __shared__ float s_inv[COLS ? 128 : 1];
    __shared__ uint32_t s_block[8];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cl = threadIdx.x & 15, rl = threadIdx.x >> 4;
    const int col0 = blockIdx.x * 128, col = col0 + cl * 8;
    const int64_t batch = blockIdx.z;
    const char *x = static_cast<const char *>(p.x) + batch * p.x_batch * (BF16 ? 2 : 4);
    const int tiles_y = (p.rows + TR - 1) / TR;
    for (int ty = blockIdx.y; ty < tiles_y; ty += gridDim.y) {
        const int row0 = ty * TR + rl;
        uint32_t v[N][W];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = row0 + 16 * i;
            if (row < p.rows) {
                load8<BF16>(p, x + static_cast<int64_t>(row) * p.ldx * (BF16 ? 2 : 4), col, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[i][j] = 0u;
            }
        }
        // the thread's amax by column, which also says whether there is an infinity
        uint32_t cm[W], any = 0u;
        auto columns = [&]() {
            any = 0u;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                cm[j] = 0u;
#pragma unroll
                for (int i = 0; i < N; ++i) cm[j] = amax_word<BF16>(cm[j], v[i][j]);
                any = max(any, amax_bits_of<BF16>(cm[j]));
            }
        };
        columns();
        if (any == kInf) {
            drop_infinities<BF16, N>(v);
            columns();
        }
        if constexpr (MODE == 1 || MODE == 3) {
            const int gi = blockIdx.x;
            const bool last = col0 + 128 >= p.cols;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                uint32_t m = 0u;
#pragma unroll
                for (int j = 0; j < W; ++j) m = amax_word<BF16>(m, v[i][j]);
                uint32_t amax = amax_bits_of<BF16>(m);
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                const int row = row0 + 16 * i;
                const uint32_t byte = ue8m0_of_amax(amax);
                if (row < p.rows) put_codes<BF16>(p, p.q + static_cast<int64_t>(row) * p.ldq, col, v[i], inv_scale(byte));
                if (cl == 0 && row < p.sf_ld)   // (rows that pad the words to a multiple of 4: zero)
                    put_byte(p.sf + (static_cast<int64_t>(gi >> 2) * p.sf_ld + row) * 4, gi & 3, row < p.rows ? byte : 0u, last);
            }
        }
        if constexpr (COLS) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                cm[j] = amax_word<BF16>(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 16));
                if (lane < 16) s_col[warp][cl * W + j] = cm[j];
            }
            __syncthreads();
            if (threadIdx.x < 16 * W) {
                uint32_t m = 0u;
#pragma unroll
                for (int w = 0; w < 8; ++w) m = amax_word<BF16>(m, s_col[w][threadIdx.x]);
#pragma unroll
                for (int e = 0; e < (BF16 ? 2 : 1); ++e) {
                    const int lc = static_cast<int>(threadIdx.x) * (BF16 ? 2 : 1) + e, c = col0 + lc;
                    const uint32_t byte = ue8m0_of_amax(BF16 ? (e ? m & 0xFFFF0000u : m << 16) : m);
                    s_inv[lc] = inv_scale(byte);
                    if (c < p.sfk_ld) {
                        int word, at;
                        bool last;
                        packed_row(p, t, ty, word, at, last);
                        put_byte(p.sfk + (static_cast<int64_t>(word) * p.sfk_ld + c) * 4, at, c < p.cols ? byte : 0u, last);
                    }
                }
            }
            __syncthreads();
            float inv[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) inv[j] = s_inv[cl * 8 + j];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int row = row0 + 16 * i;
                if (row < p.rows) put_codes<BF16>(p, p.qk + static_cast<int64_t>(row) * p.ldqk, col, v[i], inv);
            }
            // (the next tile's writes to s_col and s_inv come after its own first barrier, or, s_col,
            // after every thread has passed this tile's second)
        }
        if constexpr (MODE == 4) {
            uint32_t m = __reduce_max_sync(0xFFFFFFFFu, any);
            if (lane == 0) s_block[warp] = m;
            __syncthreads();
            m = s_block[0];
#pragma unroll
            for (int w = 1; w < 8; ++w) m = max(m, s_block[w]);
            const uint32_t byte = ue8m0_of_amax(m);
            uint8_t *q = p.q + batch * p.q_batch;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int row = row0 + 16 * i;
                if (row < p.rows) put_codes<BF16>(p, q + static_cast<int64_t>(row) * p.ldq, col, v[i], inv_scale(byte));
            }
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
            if (gridDim.y < tiles_y) __syncthreads();   // s_block is free for the next tile
        }
    }
}

template <bool BF16, int MODE, int TR>
cudaError_t launch_one(const QuantParams &p, const KGroupRows &t, int batch, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const int ty = (p.rows + TR - 1) / TR;
    cfg.gridDim = dim3((p.cols + 127) / 128, ty < 65535 ? ty : 65535, batch);
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dg_quantize_kernel<BF16, MODE, TR>, p, t);
}

template <bool BF16>
cudaError_t launch_typed(const QuantParams &p, const KGroupRows &t, int batch, int mode, int num_sms, cudaStream_t stream) {
    switch (mode) {
        case 1: {
            // rows alone: tiles of 128 rows keep 8 loads a thread in flight; where they are fewer than
            // two an SM, tiles of 16 rows
            const int64_t tiles = static_cast<int64_t>((p.cols + 127) / 128) * ((p.rows + 127) / 128);
            if (tiles < 2 * num_sms) return launch_one<BF16, 1, 16>(p, t, batch, stream);
            return launch_one<BF16, 1, 128>(p, t, batch, stream);
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
