// Products of a few bf16 rows with FP4 or FP8 weights, and the two kernels of the MoE
// layer for few tokens, on the block-scaled tensor cores.
//
// The weights are the MMA's 128-row operand, straight from their packed form, their UE8M0
// scales going to TMEM as they are, so no instruction touches a weight.  The activations are
// the narrow operand: each value x of a group of 32 along K is split into pieces of the
// weights' width or less, which occupy adjacent columns and are added at the end:
//  - two E4M3 pieces, x = s (hi + lo / 16), s = 2^(floor(log2 max|x|) - 7).  hi holds 4 significant
//    bits and lo the 4 that follow (with its sign, 9 bits in all), so a bf16 value is
//    represented exactly down to 2^-13 of its group's largest, and to 2^-21 of the largest
//    below that.  An FP32 value (the layer's inner activations) has a third piece, lo2 / 256: it
//    is rounded to 14 bits down to 2^-13 of its group's largest, to 2^-25 of the largest below (rounded to
//    the 9 bits of two pieces, a layer's bf16 outputs differ from the FP32 form's by 7e-4 of their
//    size with FP8 weights and 1.5e-3 with FP4's; with 14 bits by 1e-4 and 2e-4).
//  - for FP4 weights and at most 8 rows, eight E2M1 digits, x = s sum_j d_j / 8^j with
//    s = 2^(floor(log2 max|x|) - 1): |d| <= 4, each step leaves at most 1/8 of its range, and the
//    whole is exact to 2^-23 of the group's largest (to 2^-128 absolute, for groups below 2^-105).
// Products and sums are FP32 in TMEM.
//
// With M = 128 weight rows an MMA takes as long as its 4 KB of weights take to be read from
// shared memory up to N = 64 columns, which is a third of the time they take from HBM: the
// weight stream is the bound.  The digits exist for that stream: FP4 x FP4 takes the weights
// packed, 128 bytes a row, and TMA brings them at the rate of bytes; beside E4M3 they have to
// be unpacked to a byte a code, which TMA does at 38 GB/s an SM (214 ns for 128 rows of 64
// bytes, measured with nothing but loads).
//
// A CTA computes tiles of HALVES x 128 weight rows, over K-blocks of 128 K (digits: 256 K, 128
// bytes of a row in either case):
//   warp 0      producer: weights by TMA (a 3-D box that takes weight row 4l + c to
//               operand row 32c + l, so that 128 consecutive scale words are already in
//               the order in which tcgen05.cp takes them to TMEM), scales by bulk copy.
//   warp 1      TMEM owner, MMA issuer (of the first half; warp 6 of the second: the
//               wait, scale copies, MMAs and commit of a K-block take one warp about 330
//               cycles, 490 with a branch around what one lane issues).
//   warps 2..5  epilogue, one TMEM lane quadrant each.
//   the rest    the narrow operand.
// Many tiles, and the layer's up kernel: the CTAs are persistent and take tiles in turn, the
// ring of K-blocks running on across them.  Few tiles: one tile per cluster, K split over its CTAs.  Each CTA writes its
// FP32 partial results into the shared memory of the CTA that puts them out, whose barrier
// counts their bytes (a cluster barrier in its place took 0.4 us more at 1 x 2112 x 7168),
// and which adds them in rank order: no workspace, no atomics, a fixed order.
//
// Where the pieces come from: kGemv and kUpSelf, for the fewest rows, split the activations
// themselves, four warps (kGemv with more rows: pairs) taking K-blocks in turn.  The other modes read an image of the narrow
// operand that is already in the shared-memory form of each K-block (rows of 128 bytes
// in 128-byte swizzle, and the scale words in tcgen05.cp order), two bulk copies a block:
//   kGemvPre  dg_few_split_kernel has written the image of all rows.
//   kUp       the gate and up rows of one expert (HALVES = 2) for a segment, up to `cap`
//           of the tokens routed to it; dg_layer_split_kernel has written the segments'
//           images.  The epilogue is w silu(g) u (w the routing weight), split again
//           and written as the image that kDown reads.  kUpSelf: the same without an image.
//   kDown     K runs over all segments; the accumulators of a segment are added to the
//           FP32 results of its tokens, columns of their own in TMEM, while the next
//           segment's products run.
//
// Measured, calls in a row in a graph, on weights that are not in L2 (rate: bytes of codes and
// scales, of the 6681 GB/s that a copy reaches):
//   FP4 131064 x 7168: 1 row 76 us (6.6 TB/s), 8 rows 78, 16 rows 84, 64 rows 105 us; the DRAM
//   traffic is the weights' and the output's alone.  FP8 65536 x 7168: 1 row 72, 16 rows 76 us.
//   Small products are bound by the chain of latencies from the end of one kernel to the next
//   one's last store: 1 x 1024 x 1024 3.3 us, 1 x 2112 x 7168 FP4 4.4 us.
//   MoE layer, top 8 of 64 experts, 7168 x 2048 FP4: 1 token 37.3 us (187 MB), 16 tokens 213,
//   64 tokens 256 us (1.5 GB, 5.8 TB/s).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dg_internal.h"
#include "ptx.cuh"

namespace dg {

enum FewMode : int { kGemv = 0, kGemvPre = 1, kUp = 2, kUpSelf = 3, kDown = 4 };
// Modes whose CTAs split the activations themselves.
__host__ __device__ constexpr bool splits_itself(int mode) { return mode == kGemv || mode == kUpSelf; }
__host__ __device__ constexpr bool is_up(int mode) { return mode == kUp || mode == kUpSelf; }

// The weights' form.
enum FewFormat : int {
    kFp8 = 0,        // E4M3, activations in two E4M3 pieces
    kFp4 = 1,        // E2M1 unpacked by TMA, activations in two E4M3 pieces
    kFp4Packed = 2   // E2M1 packed, activations in eight E2M1 digits
};
// Columns of a token, and 512-byte blocks of scale words per K-block and 128 rows.
__host__ __device__ constexpr int pieces_of(int w) { return w == kFp4Packed ? 8 : 2; }
__host__ __device__ constexpr int inner_pieces(int w) { return w == kFp4Packed ? 8 : 3; }   // of the layer's inner activations
__host__ __device__ constexpr int scale_blocks(int w) { return w == kFp4Packed ? 2 : 1; }
__host__ __device__ constexpr int block_k(int w) { return w == kFp4Packed ? 256 : 128; }

struct FewArgs {
    const uint16_t *x;      // kGemv, kUpSelf: bf16 activations
    int64_t ldx;
    const uint8_t *image;   // the other modes: the narrow operand's image, and its scale blocks
    const uint8_t *image_sf;
    uint8_t *out_image;     // kUp
    uint8_t *out_image_sf;
    const uint32_t *sf;     // packed scale words of the weights
    int64_t sf_expert;      // words per expert
    int sf_ld;              // words per slice
    int rows;               // weight rows of one expert (kUp: 2 i)
    int tokens;
    int kblocks;            // K-blocks of one expert
    int slices;             // scale slices of one expert's weights (packed FP4: K / 128)
    int last_mmas;          // packed FP4: MMAs of K = 64 in the last K-block (4, or 2)
    int cap;                // tokens of a segment at most (8, 16, 32; rows of a product: or 64)
    int stages;
    int out_bytes;          // room of its own for the results, or 0: split results go to the ring
    int ahead;              // kGemv: K-blocks per CTA to bring to L2 before the wait
    int accs;               // accumulator sets (1 or 2)
    int parts;              // kDown: parts of an expert's K-blocks that different CTAs of a cluster take
    int tmem_cols;
    int row_tiles;          // tiles over the weight rows (kUp: of h's columns)
    // MoE
    const int32_t *ids;
    const float *weights;
    int experts, topk, inner;   // inner: i
    // output
    const void *c;
    int64_t ldc;
    void *d;
    int64_t ldd;
    int f32;
    int32_t *status;
    uint64_t timeout_ns;
    uint32_t debug_flags;
    int b_rows;             // of the narrow operand, in shared memory
    int launches;           // kernels of the call (host only)
};

struct FewConfig {
    static constexpr int kFirstEpi = 2;
    static constexpr int first_b(int halves) { return halves == 2 ? 7 : 6; }
    // kGemv: with rows for more than one, two warps share a K-block's between them (8 x 4096 x
    // 7168 FP8 10.2 us with one, 8.3 with two; 2 x 7168 x 16384 FP4 13.3 and 12.8).
    static constexpr int members(int w, int mode, int tokens) {
        return mode == kGemv && tokens > 256 / block_k(w) ? 2 : 1;
    }
    static constexpr int b_warps(int w, int mode, int tokens) {
        return splits_itself(mode) ? 4 * members(w, mode, tokens) : 1;
    }
    static constexpr int threads(int w, int halves, int mode, int tokens = kMaxFewRows) {
        return 32 * (first_b(halves) + b_warps(w, mode, tokens));
    }
    static constexpr int kAlign = 1024;
    static constexpr int kBarBytes = 512;
    static constexpr int kMaxStages = 24;
    // Rows of the narrow operand for up to `tokens` tokens: whole MMA column steps.
    static int b_rows(int pieces, int tokens) { return (pieces * tokens + 15) / 16 * 16; }
    static int stage_bytes(int w, int halves, int b_rows) {
        return halves * 16384 + b_rows * 128 + (halves + 1) * 512 * scale_blocks(w);
    }
    // Two buffers of 8 tokens' FP32 results; of a split tile, what this CTA puts out (rows of
    // 32 items of 4 results, shared out to the cluster's CTAs) from each of its CTAs.
    static int out_bytes(int halves, int mode, int cols, int split) {
        if (split == 1) return 2 * 8 * (is_up(mode) ? 128 : halves * 128) * 4;
        return (cols * halves + split - 1) / split * split * 32 * 4 * 4;
    }
    static int fixed_bytes(int tables) { return kAlign + kBarBytes + tables; }   // beside the ring and the results
};

// Four scaled values to their E4M3 codes; what is left of them, times 16.
__device__ __forceinline__ uint32_t next_piece4(float &f0, float &f1, float &f2, float &f3) {
    const uint32_t h01 = cvt_e4m3x2(f0, f1), h23 = cvt_e4m3x2(f2, f3);
    const uint32_t b01 = e4m3x2_to_f16x2(h01), b23 = e4m3x2_to_f16x2(h23);
    const float2 g01 = __half22float2(*reinterpret_cast<const __half2 *>(&b01));
    const float2 g23 = __half22float2(*reinterpret_cast<const __half2 *>(&b23));
    f0 = (f0 - g01.x) * 16.0f;
    f1 = (f1 - g01.y) * 16.0f;
    f2 = (f2 - g23.x) * 16.0f;
    f3 = (f3 - g23.y) * 16.0f;
    return h01 | (h23 << 16);
}

// Scale of the j-th piece.  e8: biased exponent of a group's largest magnitude, kept where the scales
// are representable; 255 marks an infinity or a NaN in the group, whose scales become NaN.
__device__ __forceinline__ uint32_t piece_scale(uint32_t e8, int j) { return e8 == 255u ? 255u : e8 - 7u - 4u * j; }
constexpr uint32_t least_piece_exponent(int pieces) { return 7u + 4u * (pieces - 1); }
__device__ __forceinline__ float inverse_scale(uint32_t e8) { return __uint_as_float((261u - e8) << 23); }

// Biased exponent of the largest of a group of 32, 8 bf16 values in each of 4 lanes.
__device__ __forceinline__ uint32_t group_exponent(const uint4 &v) {
    const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    uint32_t m = max(m2 >> 16, m2 & 0xFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return m >> 7;
}
__device__ __forceinline__ void scaled(const uint4 &v, float by, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16) * by;
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * by;
    }
}

// A lane's 8 bf16 values to their pieces; returns the group's exponent.
__device__ __forceinline__ uint32_t split_bf16(const uint4 &v, uint2 &hi, uint2 &lo) {
    const uint32_t e8 = max(group_exponent(v), least_piece_exponent(2));
    float f[8];
    scaled(v, inverse_scale(e8), f);
    hi = make_uint2(next_piece4(f[0], f[1], f[2], f[3]), next_piece4(f[4], f[5], f[6], f[7]));
    lo = make_uint2(next_piece4(f[0], f[1], f[2], f[3]), next_piece4(f[4], f[5], f[6], f[7]));
    return e8;
}

// N scaled values (|f| < 4) to their j-th digits, N codes of 4 bits; what is left of them, times 8.
template <int N>
__device__ __forceinline__ uint32_t next_digits(float (&f)[N]) {
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint32_t c = cvt_e2m1x2(f[i], f[i + 1]);
        const uint32_t back = e2m1x2_to_f16x2(c);
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&back));
        code |= c << (4 * i);
        f[i] = (f[i] - v.x) * 8.0f;
        f[i + 1] = (f[i + 1] - v.y) * 8.0f;
    }
    return code;
}
__device__ __forceinline__ uint32_t digit_scale(uint32_t e8, int j) { return e8 == 255u ? 255u : e8 - 1u - 3u * j; }
__device__ __forceinline__ float inverse_digit_scale(uint32_t e8) { return __uint_as_float((255u - e8) << 23); }
constexpr uint32_t kLeastDigitExponent = 22;   // the last digit's scale is representable

// Position of operand row n's scale word in a 512-byte block (tcgen05.cp order).
__device__ __forceinline__ uint32_t sf_word(uint32_t n) { return (n & 31u) * 4u + (n >> 5); }

// Image of n tokens' K-block: their rows in units of 8 (1024 bytes).
__host__ __device__ constexpr int image_units(int pieces, int tokens) { return (pieces * tokens + 7) >> 3; }
// Units of the inner activations before segment z, whose first entry is `first` (a bound of the sum of
// the segments' own units, each of which may be rounded up).
__host__ __device__ constexpr int inner_units_before(int w, int first, int z) {
    return w == kFp4Packed ? first : inner_pieces(w) * first / 8 + z;
}

// The lanes of one row's K-block (16, digits: 32; lane q holds values 8 q ..) write token column
// col of the K-block's image and its scales.  All lanes of a warp come here; `in`: to write.
template <int W>
__device__ __forceinline__ void split_row(const uint4 &v, uint8_t *image, uint8_t *sf, int col, int q, bool in) {
    if constexpr (W != kFp4Packed) {
        uint2 hi, lo;
        const uint32_t e8 = split_bf16(v, hi, lo);
        if (!in) return;
        const uint32_t n = 2 * col;
        const uint32_t off = (q & 1) * 8;
        *reinterpret_cast<uint2 *>(image + n * 128 + (((q >> 1) ^ (n & 7)) << 4) + off) = hi;
        *reinterpret_cast<uint2 *>(image + (n + 1) * 128 + (((q >> 1) ^ ((n + 1) & 7)) << 4) + off) = lo;
        if ((q & 3) == 0) {
            uint8_t *s = sf + sf_word(n) * 4 + (q >> 2);
            s[0] = static_cast<uint8_t>(piece_scale(e8, 0));
            s[16] = static_cast<uint8_t>(piece_scale(e8, 1));
        }
    } else {
        const uint32_t e8 = max(group_exponent(v), kLeastDigitExponent);
        float f[8];
        scaled(v, inverse_digit_scale(e8), f);
        uint8_t *s = sf + (q >> 4) * 512 + sf_word(8 * col) * 4 + ((q >> 2) & 3);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t code = next_digits(f);
            if (!in) continue;
            *reinterpret_cast<uint32_t *>(image + (8 * col + j) * 128 + (((q >> 2) ^ j) << 4) + (q & 3) * 4) = code;
            if ((q & 3) == 0) s[16 * j] = static_cast<uint8_t>(digit_scale(e8, j));
        }
    }
}

// Splits all rows of a product once for all CTAs that read them.
template <int W>
__global__ void __launch_bounds__(256) dg_few_split_kernel(const uint16_t *x, int64_t ldx, int rows, int k,
                                                           uint8_t *image, uint8_t *image_sf) {
    constexpr int LANES = block_k(W) / 8;
    grid_dependency_wait();
    grid_launch_dependents();   // after the wait: the next kernel may read what was there before this one
    const int unit = blockIdx.x * (256 / LANES) + static_cast<int>(threadIdx.x) / LANES;
    const int q = threadIdx.x % LANES;
    const bool in = unit < rows * ((k + block_k(W) - 1) / block_k(W));
    const int kb = in ? unit / rows : 0, t = in ? unit % rows : 0;
    const int at = kb * block_k(W) + q * 8;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (at < k) v = __ldcg(reinterpret_cast<const uint4 *>(x + t * ldx + at));
    __syncwarp();
    split_row<W>(v, image + static_cast<int64_t>(kb) * image_units(pieces_of(W), rows) * 1024,
                 image_sf + static_cast<int64_t>(kb) * scale_blocks(W) * 512, t, q, in);
}

// The layer's routing, as every CTA of its kernels derives it from the ids (in shared
// memory; the same in all of them): the tokens of each expert in use form one segment
// after another of up to `cap` tokens.
struct Segments {
    int count, entries;
    uint16_t *expert;   // [count]
    uint16_t *first;    // [count] first entry
    uint16_t *tokens;   // [count]
    uint16_t *unit;     // [count] units of the segments before (image_units)
    uint16_t *token;    // [entries] by expert, ascending
    uint16_t *of_entry; // [entries] segment
    uint16_t *id;       // [pairs] expert of a slot, 0xFFFF where none
    float *weight;      // [pairs] its routing weight, where asked for
};

__host__ __device__ constexpr int segment_table_bytes(int pairs, int experts) {
    const int masks = experts < 3 ? 32 : 12 * experts;   // either form's tables by expert
    return (16 + masks + 18 * pairs + 15) / 16 * 16;
}

// (The loops are not unrolled: a kernel's first pass over its code waits for the code, from
// HBM where the weights have pushed it out of L2.)
// Tables for up to 8 tokens, where an expert's tokens are one segment: a bit for each token
// and expert, from which every slot counts the entries and segments before its own.
__device__ __forceinline__ Segments build_short_segments(int *tab, const int32_t *ids, const float *weights, int id,
                                                         float weight, int tokens, int topk, int experts, int pieces,
                                                         int32_t *status) {
    const int words = (experts + 31) / 32, pairs = tokens * topk;
    uint32_t *mask = reinterpret_cast<uint32_t *>(tab + 4);   // [words][8 tokens]
    Segments s;
    s.weight = reinterpret_cast<float *>(mask + 8 * words);
    s.id = reinterpret_cast<uint16_t *>(s.weight + pairs);
    s.token = s.id + pairs;
    s.of_entry = s.token + pairs;
    s.expert = s.of_entry + pairs;
    s.first = s.expert + pairs;
    s.tokens = s.first + pairs;
    s.unit = s.tokens + pairs;
#pragma unroll 1
    for (int i = threadIdx.x; i < 8 * words; i += blockDim.x) mask[i] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int q = threadIdx.x; q < pairs; q += blockDim.x) {
        const bool mine = q == static_cast<int>(threadIdx.x);
        const int t = q / topk, e = mine ? id : __ldcg(ids + q);
        const bool ok = e >= 0 && e < experts;
        if (ok) atomicOr(&mask[(e >> 5) * 8 + t], 1u << (e & 31));
        else if (e >= experts && status) atomicOr(status, DG_DEV_BAD_GROUP);
        s.id[q] = ok ? static_cast<uint16_t>(e) : 0xFFFFu;
        if (weights) s.weight[q] = mine ? weight : __ldcg(weights + q);
    }
    __syncthreads();
    // (the last thread counts all of them)
#pragma unroll 1
    for (int q = threadIdx.x; q < pairs || threadIdx.x == blockDim.x - 1; q += blockDim.x) {
        const int t = q / topk, e = q < pairs ? s.id[q] : 32 * words;
        if (e == 0xFFFF) continue;
        int first = 0, z = 0;
        uint32_t have = 0;   // the tokens that name e
#pragma unroll 1
        for (int w = 0; w <= min(e >> 5, words - 1); ++w) {
            const uint4 a = *reinterpret_cast<const uint4 *>(mask + 8 * w), b = *reinterpret_cast<const uint4 *>(mask + 8 * w + 4);
            const uint32_t m[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            const uint32_t before = w == e >> 5 ? (1u << (e & 31)) - 1u : ~0u;
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                any |= m[i];
                first += __popc(m[i] & before);
                have = (have & ~(1u << i)) | (m[i] >> (e & 31) & 1u) << i;
            }
            z += __popc(any & before);
        }
        if (q >= pairs) {
            tab[0] = z;
            tab[1] = first;
            break;
        }
        // (a token that names an expert twice writes the same entry twice)
        const int at = __popc(have & ((1u << t) - 1u));
        s.token[first + at] = static_cast<uint16_t>(t);
        s.of_entry[first + at] = static_cast<uint16_t>(z);
        if (at == 0) {
            s.expert[z] = static_cast<uint16_t>(e);
            s.first[z] = static_cast<uint16_t>(first);
            s.tokens[z] = static_cast<uint16_t>(__popc(have));
            s.unit[z] = static_cast<uint16_t>(pieces == 8 ? first : z * image_units(pieces, tokens));
        }
    }
    __syncthreads();
    s.count = tab[0];
    s.entries = tab[1];
    return s;
}

// Tables of segment_table_bytes at `tab`; called by all threads of a CTA, after some work of
// its own if it has any (`id`, `weight`: loads of thread q's slot q, issued before that).
__device__ __forceinline__ Segments build_segments(int *tab, const int32_t *ids, const float *weights, int id, float weight,
                                                   int tokens, int topk, int experts, int cap, int pieces,
                                                   int32_t *status) {
    if (tokens <= 8)
        return build_short_segments(tab, ids, weights, id, weight, tokens, topk, experts, pieces, status);
    const int pairs = tokens * topk;
    uint32_t *mask = reinterpret_cast<uint32_t *>(tab + 4);            // [experts][2] tokens of each expert
    uint16_t *start = reinterpret_cast<uint16_t *>(mask + 2 * experts);   // [experts] first entry
    uint16_t *seg0 = start + experts;                                     // [experts] first segment
    Segments s;
    s.weight = reinterpret_cast<float *>(seg0 + experts);
    s.id = reinterpret_cast<uint16_t *>(s.weight + pairs);
    s.token = s.id + pairs;
    s.of_entry = s.token + pairs;
    s.expert = s.of_entry + pairs;
    s.first = s.expert + pairs;
    s.tokens = s.first + pairs;
    s.unit = s.tokens + pairs;
    const int lane = threadIdx.x & 31;
    const int shift = __ffs(cap) - 1;   // (a power of two; runtime divisions would cost over a microsecond here)
#pragma unroll 1
    for (int e = threadIdx.x; e < 2 * experts; e += blockDim.x) mask[e] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int q = threadIdx.x; q < pairs; q += blockDim.x) {
        const bool mine = q == static_cast<int>(threadIdx.x);
        const int e = mine ? id : __ldcg(ids + q);
        const bool ok = e >= 0 && e < experts;
        if (e >= experts && status) atomicOr(status, DG_DEV_BAD_GROUP);
        s.id[q] = ok ? static_cast<uint16_t>(e) : 0xFFFFu;
        if (weights) s.weight[q] = mine ? weight : __ldcg(weights + q);
        const int t = q / topk;
        if (ok) atomicOr(&mask[2 * e + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        // lane l counts experts l * per .., one scan over the lanes, then it lays out its segments
        const int per = (experts + 31) / 32, full = image_units(pieces, cap);
        // (trip counts are the same in all lanes: shuffles after a loop that could diverge take
        // 270 cycles each)
        int n = 0, segs = 0, units = 0;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            const int c = e < experts ? __popc(mask[2 * e]) + __popc(mask[2 * e + 1]) : 0;
            n += c;
            segs += (c + cap - 1) >> shift;
            units += (c >> shift) * full + image_units(pieces, c & (cap - 1));
        }
        __syncwarp();
        int in_n = n, in_su = segs | units << 16;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, in_n, d), v = __shfl_up_sync(0xFFFFFFFFu, in_su, d);
            in_n += lane >= d ? u : 0;
            in_su += lane >= d ? v : 0;
        }
        int first = in_n - n, z = (in_su & 0xFFFF) - segs, u = (in_su >> 16) - units;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e >= experts) continue;
            start[e] = static_cast<uint16_t>(first);
            seg0[e] = static_cast<uint16_t>(z);
#pragma unroll 1
            for (int left = __popc(mask[2 * e]) + __popc(mask[2 * e + 1]); left > 0; left -= cap, ++z) {
                const int t = min(left, cap);
                s.expert[z] = static_cast<uint16_t>(e);
                s.first[z] = static_cast<uint16_t>(first);
                s.tokens[z] = static_cast<uint16_t>(t);
                s.unit[z] = static_cast<uint16_t>(u);
                first += t;
                u += image_units(pieces, t);
            }
        }
        if (lane == 31) { tab[0] = in_su & 0xFFFF; tab[1] = in_n; }
    }
    __syncthreads();
#pragma unroll 1
    for (int q = threadIdx.x; q < pairs; q += blockDim.x) {
        const int e = s.id[q], t = q / topk;
        if (e == 0xFFFF) continue;
        // (a token that names an expert twice writes the same entry twice)
        const uint32_t below = (1u << (t & 31)) - 1u;
        const int at = t < 32 ? __popc(mask[2 * e] & below) : __popc(mask[2 * e]) + __popc(mask[2 * e + 1] & below);
        s.token[start[e] + at] = static_cast<uint16_t>(t);
        s.of_entry[start[e] + at] = static_cast<uint16_t>(seg0[e] + (at >> shift));
    }
    __syncthreads();
    s.count = tab[0];
    s.entries = tab[1];
    return s;
}

// Images of all segments' tokens.  Blocks of grid.y take entries in turn, one K-block each.
template <int W>
__global__ void __launch_bounds__(256) dg_layer_split_kernel(const uint16_t *x, int64_t ldx, const int32_t *ids,
                                                             int tokens, int topk, int experts, int cap, int k,
                                                             uint8_t *image, uint8_t *image_sf) {
    constexpr int LANES = block_k(W) / 8, ROWS = 256 / LANES;
    extern __shared__ int split_tab[];
    // x's part to L2 meanwhile (which makes no difference to what is read later)
    if (blockIdx.y == 0 && static_cast<int>(threadIdx.x) < tokens)
        prefetch_l2_bulk(x + threadIdx.x * ldx + blockIdx.x * block_k(W),
                         2 * min(block_k(W), k - static_cast<int>(blockIdx.x) * block_k(W)));
    grid_dependency_wait();
    grid_launch_dependents();
    const int slot_id = threadIdx.x < tokens * topk ? __ldcg(ids + threadIdx.x) : -1;
    const Segments s = build_segments(split_tab, ids, nullptr, slot_id, 0.0f, tokens, topk, experts, cap, pieces_of(W), nullptr);
    const int q = threadIdx.x % LANES, kb = blockIdx.x, kblocks = gridDim.x;
    const int col = kb * block_k(W) + q * 8;
    for (int at0 = blockIdx.y * ROWS; at0 < s.entries; at0 += gridDim.y * ROWS) {
        const int at = at0 + static_cast<int>(threadIdx.x) / LANES;
        const bool in = at < s.entries;
        const int row = in ? s.token[at] : 0, z = in ? s.of_entry[at] : 0;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (col < k) v = __ldcg(reinterpret_cast<const uint4 *>(x + row * ldx + col));
        const int units = image_units(pieces_of(W), s.tokens[z]);
        __syncwarp();
        split_row<W>(v, image + (static_cast<int64_t>(s.unit[z]) * kblocks + kb * units) * 1024,
                     image_sf + (static_cast<int64_t>(z) * kblocks + kb) * scale_blocks(W) * 512, at - s.first[z], q, in);
    }
}

// One tile of work, the same for every role of a CTA.
struct FewTile {
    int seg;        // kUp
    int expert;     // kUp
    int row0;       // first weight row (kUp: column of h)
    int ntok;       // token columns (kDown: all tokens)
};

// A CTA's K-blocks of a run: kb, kb + 1, ..
struct FewRun {
    int kb, n;
};

template <int W, int HALVES, int MODE>
__global__ void __launch_bounds__(FewConfig::threads(W, HALVES, MODE), is_up(MODE) ? 1 : 2)
    dg_few_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ FewArgs p) {
    constexpr bool UP = is_up(MODE), SELF = splits_itself(MODE);
    constexpr int ROWS = HALVES * 128;
    constexpr int OUT = UP ? 128 : ROWS;     // results per token and tile
    constexpr int FIRST_B = FewConfig::first_b(HALVES);
    constexpr bool DIGITS = W == kFp4Packed;
    const int members = FewConfig::members(W, MODE, p.tokens);
    constexpr int INNER = inner_pieces(W), PIECES = MODE == kDown ? INNER : pieces_of(W);
    constexpr int SB = scale_blocks(W), BLOCK_K = block_k(W);
    constexpr int SF = 4 * SB + 4 * SB;               // TMEM columns of a K-block's scales: weights', activations'
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int rank = UP ? 0 : static_cast<int>(cluster_ctarank());
    const int nsplit = UP ? 1 : static_cast<int>(cluster_nctarank());
    const int S = p.stages;
    const int ncols = (PIECES * p.cap + 15) & ~15;
    const int b_bytes = p.b_rows * 128;
    uint8_t *smem_a = smem;
    uint8_t *smem_b = smem_a + S * HALVES * 16384;
    uint8_t *smem_sfa = smem_b + S * b_bytes;
    uint8_t *smem_sfb = smem_sfa + S * HALVES * SB * 512;
    uint8_t *smem_end = smem_sfb + S * SB * 512;
    float *smem_out = reinterpret_cast<float *>(p.out_bytes ? smem_end : smem_a);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem_end + p.out_bytes);
    uint64_t *full_bar = bars;              // [S] weights and scales landed, pieces landed or written
    uint64_t *empty_bar = bars + S;         // [S] the slot's MMAs are done
    uint64_t *tfull_bar = bars + 2 * S;     // [2] accumulators complete
    uint64_t *tempty_bar = tfull_bar + 2;   // [2] accumulators read
    uint64_t *drain_bar = tempty_bar + 2;   // [HALVES]
    uint64_t *join_bar = drain_bar + HALVES;   // split tiles: the results that this CTA puts out are here
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(join_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *tab = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + FewConfig::kBarBytes);

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0);   // (known to be the same in a warp)
    const int lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};
    const int first_tile = blockIdx.x / nsplit, tile_step = gridDim.x / nsplit;

    const int pairs = MODE < kUp ? 0 : p.tokens * p.topk;
    // (kUpSelf is the first kernel of its call: its ids may be the preceding kernel's)
    int slot_id = -1;
    float slot_weight = 0.0f;
    auto load_slot = [&] {
        if (static_cast<int>(threadIdx.x) >= pairs) return;
        slot_id = __ldcg(p.ids + threadIdx.x);
        if constexpr (UP) slot_weight = __ldcg(p.weights + threadIdx.x);
    };
    if constexpr (MODE == kUp || MODE == kDown) load_slot();
    if (warp == 0) {
        // arrivals: full one for weights and `members` for pieces, empty and tfull one per issuer, tempty 4, drain 1
        for (int i = lane; i < 2 * S + 4 + HALVES + 1; i += 32)
            mbar_init(bars + i, i < S ? 1 + members : i < 2 * S + 2 ? HALVES : i < 2 * S + 4 ? 4 : 1);
        if (lane == 0) {
            *abort_flag = 0;
            tma_prefetch_desc(&tm_w);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, p.tmem_cols);
        tmem_relinquish();
    }
    __syncwarp();
    // Split tiles: the CTAs may write to a peer's shared memory once it has started or, where
    // the results go to the ring, once its ring is idle.
    const bool early = p.out_bytes != 0;
    if (nsplit > 1 && early) cluster_arrive_relaxed();
    // The kernel before kGemvPre, kUp and kDown (a split kernel or kUpSelf) waits for what
    // precedes it and only then lets the next one start.  So these may read weights, ids and
    // routing weights at once, and the warps that read the preceding kernel's output wait
    // for it.  In kGemv every warp waits that reads or writes memory, in kUpSelf all do here.
    // No timed wait begins before the preceding kernel's end, whose time is none of this one's: the
    // issuers wait for it first, the producer before it waits for a slot of the ring to be free.
    if constexpr (MODE == kUpSelf) {
        grid_dependency_wait();
        load_slot();
    }
    grid_launch_dependents();
    Segments seg = {};
    if constexpr (MODE >= kUp)
        seg = build_segments(tab, p.ids, UP ? p.weights : nullptr, slot_id, slot_weight, p.tokens, p.topk, p.experts,
                             p.cap, pieces_of(W), p.status);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    const int num_tiles = UP ? seg.count * p.row_tiles : p.row_tiles;
    // A tile's K-blocks are one run, of which each CTA of a cluster has a share; in kDown a run for
    // each segment, cut into p.parts parts that fall to CTAs by the expert alone.  (Equal
    // shares of all segments' K-blocks would make the order in which a token's products are summed
    // depend on the other tokens' experts.)
    const int runs = MODE == kDown ? seg.count : 1;
    const int k_begin = static_cast<int>(static_cast<int64_t>(p.kblocks) * rank / nsplit);
    const int k_end = static_cast<int>(static_cast<int64_t>(p.kblocks) * (rank + 1) / nsplit);
    const int part_base = MODE == kDown ? p.kblocks / p.parts : 0, part_odd = MODE == kDown ? p.kblocks % p.parts : 0;
    const uint32_t split_inv = 65536u / nsplit + 1u;
    auto run_of = [&](int z) {
        if constexpr (MODE != kDown) return FewRun{k_begin, k_end - k_begin};
        const auto mod = [&](uint32_t v) { return v - (v * split_inv >> 16) * nsplit; };   // (v below 1024)
        // part j of expert e falls to CTA e * parts + j
        int j = rank - static_cast<int>(mod(mod(seg.expert[z]) * p.parts));
        if (j < 0) j += nsplit;
        if (j >= p.parts) return FewRun{0, 0};
        return FewRun{part_base * j + min(j, part_odd), part_base + (j < part_odd ? 1 : 0)};
    };

    auto get_tile = [&](int w) {
        FewTile t = {0, 0, w * ROWS, p.tokens};
        if constexpr (UP) {
            t.seg = w / p.row_tiles;
            t.row0 = (w - t.seg * p.row_tiles) * 128;
            t.expert = seg.expert[t.seg];
            t.ntok = seg.tokens[t.seg];
        }
        return t;
    };
    // Four results of one token at weight rows n .. n + 3 (kUp: a warp holds the token's
    // 128; o is already silu(g) u).
    auto store = [&](const FewTile &tile, int t, int n, float (&o)[4]) {
        if constexpr (UP) {
            // the routing weight, summed over the token's slots that name this expert
            const int slot = seg.token[seg.first[tile.seg] + t] * p.topk + lane;
            float w = lane < p.topk && seg.id[slot] == tile.expert ? seg.weight[slot] : 0.0f;
            __syncwarp();
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, s);
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                o[c] *= w;
                m = max(m, __float_as_uint(o[c]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));   // a group of 32
            // this tile is a K-block of kDown, or half of one
            const int kblocks = (p.inner + BLOCK_K - 1) / BLOCK_K, kb = tile.row0 / BLOCK_K, k0 = tile.row0 % BLOCK_K;
            uint8_t *image = p.out_image + (static_cast<int64_t>(inner_units_before(W, seg.first[tile.seg], tile.seg)) * kblocks +
                                            kb * image_units(INNER, tile.ntok)) * 1024;
            uint8_t *sf = p.out_image_sf + ((static_cast<int64_t>(tile.seg) * kblocks + kb) * SB + k0 / 128) * 512 + (lane >> 3);
            if constexpr (DIGITS) {
                const uint32_t e8 = max(m >> 23, kLeastDigitExponent);
                const float inv = inverse_digit_scale(e8);
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] *= inv;
                const uint32_t at = k0 / 2 + lane * 2;   // byte of the row
#pragma unroll
                for (int j = 0; j < INNER; ++j) {
                    const uint32_t code = next_digits(o);
                    *reinterpret_cast<uint16_t *>(image + (INNER * t + j) * 128 + (((at >> 4) ^ j) << 4) + (at & 15)) =
                        static_cast<uint16_t>(code);
                    if ((lane & 7) == 0) sf[sf_word(INNER * t + j) * 4] = static_cast<uint8_t>(digit_scale(e8, j));
                }
            } else {
                const uint32_t e8 = max(m >> 23, least_piece_exponent(INNER));
                const float inv = inverse_scale(e8);
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] *= inv;
#pragma unroll
                for (int j = 0; j < INNER; ++j) {
                    const uint32_t r = INNER * t + j, code = next_piece4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint32_t *>(image + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) = code;
                    if ((lane & 7) == 0) sf[sf_word(r) * 4] = static_cast<uint8_t>(piece_scale(e8, j));
                }
            }
        } else if (n < p.rows) {
            if (p.f32) {
                if (p.c) {
                    const float4 c =
                        __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.c) + t * p.ldc + n));
                    o[0] += c.x; o[1] += c.y; o[2] += c.z; o[3] += c.w;
                }
                *reinterpret_cast<float4 *>(static_cast<float *>(p.d) + t * p.ldd + n) =
                    make_float4(o[0], o[1], o[2], o[3]);
            } else {
                if (p.c) {
                    const uint2 c =
                        __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.c) + t * p.ldc + n));
                    o[0] += __uint_as_float(c.x << 16);
                    o[1] += __uint_as_float(c.x & 0xFFFF0000u);
                    o[2] += __uint_as_float(c.y << 16);
                    o[3] += __uint_as_float(c.y & 0xFFFF0000u);
                }
                const __nv_bfloat162 a = __floats2bfloat162_rn(o[0], o[1]), b = __floats2bfloat162_rn(o[2], o[3]);
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.d) + t * p.ldd + n) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
            }
        }
    };
    // All warps come by once: before they push results, or with nothing left to do.
    auto ring_idle = [&] {
        if (!early) cluster_arrive();
        cluster_wait();
    };
    auto gated = [](float g, float u) { return g / (1.0f + expf(-g)) * u; };

    // TMEM columns: accumulator sets, two scale slots for each issuer, kDown's results
    const uint32_t sf_tmem = tmem_base + p.accs * HALVES * ncols;
    const uint32_t y_tmem = sf_tmem + 2 * HALVES * SF;          // [HALVES][tokens, up to 8]
    const int y_cols = (p.tokens + 7) & ~7;

    // nsplit > 1.  A tile's results are rows of 32 items, item l the 4 results
    // that lane l of the four epilogue warps hold: ROW_GROUPS rows a token.
    // CTA r puts out rows r * share .. of them; smem_out is [CTA][share][component][32].
    constexpr int ROW_GROUPS = OUT / 128, COMP = 4;
    const int share = nsplit > 1 && first_tile < num_tiles
                          ? (get_tile(first_tile).ntok * ROW_GROUPS + nsplit - 1) / nsplit : 0;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int slot = 0;
        uint32_t phase = 0;
        uint32_t issued = 0;
        bool waited = MODE == kGemv || MODE == kUpSelf;
        const bool one = elect_one();
        bool drop = (p.debug_flags & DG_DEBUG_DROP_ONE_LOAD) && blockIdx.x == 0;
        const auto box_row = [&](const FewTile &tile, int e, int h) {   // rows / 4 of a half's box
            const int r = UP ? h * p.inner + tile.row0 : tile.row0 + h * 128;
            return static_cast<int32_t>((static_cast<int64_t>(e) * p.rows + r) >> 2);
        };
        if constexpr (MODE == kGemv) {
            // The first K-blocks' weights to L2 while the preceding kernel ends (which makes no
            // difference to what is read after the wait).
            if (first_tile < num_tiles && elect_one()) {
                const FewTile tile = get_tile(first_tile);
                for (int i = k_begin; i < min(k_end, k_begin + p.ahead); ++i)
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) tma_prefetch_3d(&tm_w, i * 128, box_row(tile, 0, h), 0);
            }
            __syncwarp();
            grid_dependency_wait();
        }
        for (int w = first_tile; w < num_tiles; w += tile_step) {
            const FewTile tile = get_tile(w);
            for (int z = 0; z < runs; ++z) for (FewRun run = run_of(z); run.n > 0; ++run.kb, --run.n) {
                const int kb = run.kb;
                if (!mbar_wait_warp(&empty_bar[slot], phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto producer_done;
                if (drop) drop = false;   // diagnostic: this slot never fills
                else issued |= 1u << slot;
                const bool on = one && (issued >> slot & 1u);
                const int e = MODE == kDown ? seg.expert[z] : tile.expert;
                const int slice = W == kFp8 ? kb >> 2 : kb * SB;
                const int slices = min(SB, p.slices - slice);
                const uint32_t *sf = p.sf + e * p.sf_expert + static_cast<int64_t>(slice) * p.sf_ld;
                uint32_t sf_bytes[HALVES];
                uint32_t bytes = HALVES * (W == kFp4 ? 8192 : 16384);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const int left = UP ? 128 : p.sf_ld - (tile.row0 + h * 128);
                    sf_bytes[h] = left >= 128 ? 512u : left > 0 ? 4u * static_cast<uint32_t>(left) : 0u;
                    bytes += sf_bytes[h] * slices;
                }
                mbar_arrive_expect_tx_if(on, &full_bar[slot], bytes);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const int r = UP ? h * p.inner + tile.row0 : tile.row0 + h * 128;
                    // (a half past the last row reads zeros or the next expert's rows; unused)
                    tma_load_3d_if(on, smem_a + (slot * HALVES + h) * 16384, &tm_w, &full_bar[slot], kb * 128,
                                   box_row(tile, e, h), 0);
#pragma unroll
                    for (int b = 0; b < SB; ++b)
                        bulk_load_if(on && sf_bytes[h] && b < slices, smem_sfa + ((slot * HALVES + h) * SB + b) * 512,
                                     sf + static_cast<int64_t>(b) * p.sf_ld + r, sf_bytes[h], &full_bar[slot]);
                }
                if (++slot == S) {
                    slot = 0;
                    phase ^= 1;
                    if (!waited) grid_dependency_wait();
                    waited = true;
                }
            }
        }
    producer_done:
        __syncwarp();
        if (nsplit > 1) ring_idle();
        // Normally every load has landed once the MMAs are done.  After a wait that ran
        // out, never leave with loads in flight: give them the time limit once more.
        named_bar_sync(2, 32 + 32 * HALVES);   // the issuers are done with their waits
        if (lane == 0 && *abort_flag) {
            const uint64_t t0 = global_timer_ns();
            for (int s = 0; s < S; ++s)
                while ((issued & (1u << s)) && global_timer_ns() - t0 < ctl.timeout_ns &&
                       !mbar_try_wait(smem_u32(&full_bar[s]), s < slot ? phase : phase ^ 1)) {}
        }
        __syncwarp();
    } else if (warp == 1 || (HALVES == 2 && warp == FIRST_B - 1)) {
        // ------------------------------------------------------------ MMA issuers
        const int h = warp == 1 ? 0 : 1;
        int slot = 0, acc = 0, g = 0;
        uint32_t phase = 0, acc_phase = 0;
        const uint64_t a_base = make_desc_kmajor_sw128(smem_u32(smem_a + h * 16384));
        const uint64_t b_base = make_desc_kmajor_sw128(smem_u32(smem_b));
        const uint64_t sfa_base = make_desc_sf_32x128b(smem_u32(smem_sfa + h * SB * 512));
        const uint64_t sfb_base = make_desc_sf_32x128b(smem_u32(smem_sfb));
        const uint32_t sf0 = sf_tmem + 2 * h * SF;
        const bool one = elect_one();
        if constexpr (MODE != kUpSelf) grid_dependency_wait();   // (the narrow operand comes after it anyway)
        for (int w = first_tile; w < num_tiles; w += tile_step) {
            const FewTile tile = get_tile(w);
            // each run into one accumulator
            for (int i = 0; i < runs; ++i) {
                const FewRun run = run_of(i);
                const int z = MODE == kDown ? i : tile.seg, kb0 = run.kb, n = run.n;
                if (MODE == kDown && n == 0) continue;
                if (!mbar_wait_warp(&tempty_bar[acc], acc_phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto mma_done;
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + (acc * HALVES + h) * ncols;
                // columns in use: the tokens', rounded up to the MMA's step of 16
                const int tok = MODE >= kUp ? __shfl_sync(0xFFFFFFFFu, static_cast<int>(seg.tokens[z]), 0) : tile.ntok;
                const uint32_t cols = (PIECES * tok + 15) / 16 * 16;
                const uint32_t idesc = DIGITS ? make_idesc_mxf4(128, cols, 0, 0)
                                              : make_idesc_mxf8(128, cols, 0, 0) | (W == kFp4 ? 5u << 7 : 0u);   // A: E2M1
                // (nothing here diverges: a branch for the issuing lane costs 200 cycles a K-block)
                for (int j = 0; j < n; ++j, ++g) {
                    if (!mbar_wait_warp(&full_bar[slot], phase, ctl, DG_DEV_TIMEOUT)) goto mma_done;
                    tc_fence_after_sync();
                    const int next = slot + 1 == S ? 0 : slot + 1;
                    const uint32_t sf = sf0 + (g & 1) * SF;
#pragma unroll
                    for (int b = 0; b < SB; ++b) {
                        tc_cp_32x128b_warpx4_if(one, sf + 4 * b,
                                                sfa_base + static_cast<uint64_t>((slot * HALVES * SB + b) * 32));
                        tc_cp_32x128b_warpx4_if(one, sf + 4 * SB + 4 * b,
                                                sfb_base + static_cast<uint64_t>((slot * SB + b) * 32));
                    }
                    const uint64_t a_desc = a_base + static_cast<uint64_t>(slot * HALVES * 1024);
                    const uint64_t b_desc = b_base + static_cast<uint64_t>(slot * (b_bytes >> 4));
                    if constexpr (DIGITS) {
                        const bool all = one && (kb0 + j != p.kblocks - 1 || p.last_mmas == 4);
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) {
                            const uint32_t byte = (k & 1) * 2;   // of the slice's scale words
                            tc_mma_mxf4_if(k < 2 ? one : all, d_tmem, a_desc + 2 * k, b_desc + 2 * k,
                                           idesc | (byte << 4) | (byte << 29), sf + 4 * (k >> 1),
                                           sf + 4 * SB + 4 * (k >> 1), (j | k) != 0);
                        }
                    } else {
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) {
                            // scale byte: the activations' and FP4 weights' k-th 32 K, FP8 weights' 128-K block
                            const uint32_t id =
                                idesc | (k << 4) | ((W == kFp4 ? k : static_cast<uint32_t>((kb0 + j) & 3)) << 29);
                            tc_mma_mxf8_if(one, d_tmem, a_desc + 2 * k, b_desc + 2 * k, id, sf, sf + 4, (j | k) != 0);
                        }
                    }
                    tc_commit_if(one, &empty_bar[slot]);
                    slot = next;
                    phase ^= next == 0;
                }
                tc_commit_if(one, &tfull_bar[acc]);
                if (++acc == p.accs) { acc = 0; acc_phase ^= 1; }
            }
        }
    mma_done:
        __syncwarp();
        if (nsplit > 1) ring_idle();
        // TMEM is not freed before every MMA has finished
        tc_commit_if(one, &drain_bar[h]);
        if (one) {
            mbar_wait_drain(&drain_bar[h], 0, ctl);
        }
        __syncwarp();
        named_bar_sync(2, 32 + 32 * HALVES);
    } else if (warp >= FIRST_B) {
        // ------------------------------------------------------------ the narrow operand
        grid_dependency_wait();
        if constexpr (SELF) {
            // The warps take the K-blocks in turn, at most as many warps as ring slots: a
            // wait for the MMAs of block g - S tests one parity bit, which is unambiguous
            // only if block g - 2S is known to be done; a warp's previous block g - teams
            // implies that up to block g - teams - S.
            const int teams = S < 4 ? S : 4;
            const int bw = (warp - FIRST_B) >> (members - 1), member = (warp - FIRST_B) & (members - 1);
            constexpr int LANES = BLOCK_K / 8, AT_ONCE = 32 / LANES;   // of a row, and rows of a warp
            constexpr int STEPS = MODE == kGemv ? 2 : DIGITS ? 1 : 4;
            const int q = lane % LANES;
            int g = 0;   // K-blocks of the tiles before
            for (int w = first_tile; w < num_tiles && bw < teams; w += tile_step, g += k_end - k_begin) {
                const FewTile tile = get_tile(w);
                for (int i = (bw + teams - g % teams) % teams; i < k_end - k_begin; i += teams) {
                    const int slot = (g + i) % S;
                    if (!mbar_wait_warp(&empty_bar[slot], (((g + i) / S) & 1) ^ 1, ctl, DG_DEV_TIMEOUT)) goto b_done;
                    const int at = (k_begin + i) * BLOCK_K + q * 8;
                    for (int t0 = member * AT_ONCE; t0 < tile.ntok; t0 += STEPS * members * AT_ONCE) {
                        uint4 v[STEPS];   // the loads of some steps, then their splitting
#pragma unroll
                        for (int r = 0; r < STEPS; ++r) {
                            const int t = t0 + r * members * AT_ONCE + lane / LANES;
                            v[r] = make_uint4(0u, 0u, 0u, 0u);
                            if (t < tile.ntok && (!DIGITS || at < p.slices * 128)) {
                                const int row = UP ? seg.token[seg.first[tile.seg] + t] : t;
                                v[r] = __ldcg(reinterpret_cast<const uint4 *>(p.x + row * p.ldx + at));
                            }
                        }
                        __syncwarp();
#pragma unroll
                        for (int r = 0; r < STEPS; ++r) {
                            const int t = t0 + r * members * AT_ONCE + lane / LANES;
                            if (t0 + r * members * AT_ONCE >= tile.ntok) break;
                            split_row<W>(v[r], smem_b + slot * b_bytes, smem_sfb + slot * SB * 512, t, q, t < tile.ntok);
                            __syncwarp();
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full_bar[slot]);
                }
            }
        } else {
            int slot = 0;
            uint32_t phase = 0;
            const bool one = elect_one();
            for (int w = first_tile; w < num_tiles; w += tile_step) {
                const FewTile tile = get_tile(w);
                for (int i = 0; i < runs; ++i) for (FewRun run = run_of(i); run.n > 0; ++run.kb, --run.n) {
                    const int z = MODE == kDown ? i : tile.seg, kb = run.kb;
                    if (!mbar_wait_warp(&empty_bar[slot], phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto b_done;
                    const int tok = MODE >= kUp ? seg.tokens[z] : tile.ntok;
                    const int units = image_units(PIECES, tok);
                    const int64_t before = MODE == kDown ? inner_units_before(W, seg.first[z], z) : MODE >= kUp ? seg.unit[z] : 0;
                    const uint32_t sf_bytes = DIGITS ? 1024u : PIECES * tok < 32 ? 16u * PIECES * tok : 512u;
                    mbar_arrive_expect_tx_if(one, &full_bar[slot], units * 1024 + sf_bytes);
                    bulk_load_if(one, smem_b + slot * b_bytes, p.image + (before * p.kblocks + kb * units) * 1024,
                                 units * 1024, &full_bar[slot]);
                    bulk_load_if(one, smem_sfb + slot * SB * 512,
                                 p.image_sf + (static_cast<int64_t>(z) * p.kblocks + kb) * SB * 512, sf_bytes,
                                 &full_bar[slot]);
                    if (++slot == S) { slot = 0; phase ^= 1; }
                }
            }
        }
    b_done:
        __syncwarp();
        if (nsplit > 1) ring_idle();
    } else {
        // ------------------------------------------------------------ epilogue
        const uint32_t quad = warp & 3;
        const int id = threadIdx.x - 32 * FewConfig::kFirstEpi;   // 0..127
        int acc = 0, buf = 0;
        bool pushed = false;
        uint32_t acc_phase = 0;
        grid_dependency_wait();       // C, and memory that the output may share
        if (!UP && p.c && first_tile < num_tiles) {   // the first tile's C to L2
            const int size = p.f32 ? 4 : 2, lines = ROWS * size / 128;
            const int row0 = first_tile * ROWS;
            for (int i = id; i < p.tokens * lines; i += 128) {
                const int t = i / lines, at = i % lines * (128 / size);
                if (row0 + at < p.rows)
                    prefetch_l2_line(static_cast<const char *>(p.c) + (t * p.ldc + row0 + at) * size);
            }
        }
        // Results of this thread's operand row (of each half) for n tokens from t0, to the CTAs
        // that put them out.
        auto push = [&](const FewTile &tile, int t0, int n, const float (&r)[HALVES][8]) {
            int row = t0 * ROW_GROUPS, owner = 0;
            for (; row >= share; row -= share) ++owner;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= n) break;
#pragma unroll
                for (int g = 0; g < ROW_GROUPS; ++g) {
                    const uint32_t at = mapa_shared(
                        smem_u32(smem_out + ((rank * share + row) * COMP + quad) * 32 + lane), owner);
                    const uint32_t bar = mapa_shared(smem_u32(join_bar), owner);
                    st_async_cluster_f32(at, r[g][j], bar);
                    if (++row == share) { row = 0; ++owner; }
                }
            }
        };
        // 8 tokens' results from t0 at this thread's operand rows: the sums of their columns, the smallest first
        auto read8 = [&](int t0, int n, float (&r)[HALVES][8]) {
            const uint32_t col = tmem_base + ((quad * 32) << 16) + acc * HALVES * ncols + PIECES * t0;
            if constexpr (PIECES == 3) {   // (kDown) 24 columns
                uint32_t v[HALVES][3][8];
#pragma unroll
                for (int h = 0; h < HALVES; ++h)
#pragma unroll
                    for (int l = 0; l < 3; ++l) tmem_ld_32x32b_x8(col + h * ncols + 8 * l, v[h][l]);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
#pragma unroll
                    for (int l = 0; l < 3; ++l) reg_fence8(v[h][l]);
                    const auto at = [&](int c) { return __uint_as_float(v[h][c >> 3][c & 7]); };
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[h][j] = (at(3 * j + 2) + at(3 * j + 1)) + at(3 * j);
                }
            } else {
                constexpr int AT_ONCE = 16 / PIECES, LOADS = AT_ONCE < 8 && HALVES == 1 ? 2 : 1;   // tokens of 16 columns, loads in flight
#pragma unroll
                for (int j0 = 0; j0 < 8; j0 += LOADS * AT_ONCE) {
                    if (j0 >= n) break;
                    uint32_t v[LOADS][HALVES][16];
#pragma unroll
                    for (int l = 0; l < LOADS; ++l)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            if (l == 0 || j0 + l * AT_ONCE < n)
                                tmem_ld_32x32b_x16(col + h * ncols + PIECES * (j0 + l * AT_ONCE), v[l][h]);
                    tmem_ld_wait();
#pragma unroll
                    for (int l = 0; l < LOADS; ++l)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) {
                            reg_fence16(v[l][h]);
#pragma unroll
                            for (int j = 0; j < AT_ONCE; ++j) {
                                float sum = __uint_as_float(v[l][h][PIECES * j + PIECES - 1]);
#pragma unroll
                                for (int c = PIECES - 2; c >= 0; --c) sum += __uint_as_float(v[l][h][PIECES * j + c]);
                                r[h][j0 + l * AT_ONCE + j] = sum;
                            }
                        }
                }
            }
        };
        auto release = [&] {   // the accumulators are read
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty_bar[acc]);
            if (++acc == p.accs) { acc = 0; acc_phase ^= 1; }
        };
        // the four warps go on or give up together
        auto wait_acc = [&] {
            const bool ok = named_bar_and(1, 128, mbar_wait_warp(&tfull_bar[acc], acc_phase, ctl, DG_DEV_TIMEOUT));
            tc_fence_after_sync();
            return ok;
        };
        auto write_out = [&](const FewTile &tile, const float *src, int t0, int n) {   // n tokens from t0
            for (int q = id; q < n * (OUT / 4); q += 128) {
                const int t = q / (OUT / 4), l = q % (OUT / 4);
                float o[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = src[t * OUT + (l >> 5) * 128 + 32 * c + (l & 31)];
                store(tile, t0 + t, tile.row0 + 4 * l, o);
            }
        };
        for (int w = first_tile; w < num_tiles; w += tile_step) {
            const FewTile tile = get_tile(w);
            const int mine = quad * 32 + lane;
            if constexpr (MODE == kDown) {
                const uint32_t y0 = y_tmem + ((quad * 32) << 16);
                for (int c = 0; c < HALVES * y_cols; ++c) tmem_st_32x32b_x1(y0 + c, 0u);
                tmem_st_wait();
                for (int z = 0; z < runs; ++z) {
                    if (run_of(z).n == 0) continue;
                    if (!wait_acc()) goto epi_done;
                    const int tok = seg.tokens[z];
                    for (int t0 = 0; t0 < tok; t0 += 8) {
                        float r[HALVES][8];
                        uint32_t y[HALVES][8], at[8];
                        read8(t0, tok - t0, r);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (t0 + j >= tok) break;
                            at[j] = y0 + seg.token[seg.first[z] + t0 + j];
#pragma unroll
                            for (int h = 0; h < HALVES; ++h) y[h][j] = tmem_ld_32x32b_x1(at[j] + h * y_cols);
                        }
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (t0 + j >= tok) break;
#pragma unroll
                            for (int h = 0; h < HALVES; ++h) {
                                reg_fence1(y[h][j]);
                                tmem_st_32x32b_x1(at[j] + h * y_cols, __float_as_uint(__uint_as_float(y[h][j]) + r[h][j]));
                            }
                        }
                    }
                    tmem_st_wait();
                    release();
                }
                if (nsplit > 1) ring_idle();
                pushed = true;
                for (int t0 = 0; t0 < p.tokens; t0 += 8) {
                    const int n = min(8, p.tokens - t0);
                    float *out = smem_out + buf * 8 * OUT;
                    uint32_t y[HALVES][8];
                    float r[HALVES][8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) y[h][j] = tmem_ld_32x32b_x1(y0 + h * y_cols + t0 + j);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) {
                            reg_fence1(y[h][j]);
                            r[h][j] = __uint_as_float(y[h][j]);
                            if (j < n && nsplit == 1) out[j * ROWS + h * 128 + mine] = r[h][j];
                        }
                    }
                    if (nsplit > 1) {
                        push(tile, t0, n, r);
                        continue;
                    }
                    named_bar_sync(1, 128);
                    write_out(tile, out, t0, n);
                    buf ^= 1;
                }
            } else {
                if (!wait_acc()) break;
                if (nsplit > 1) ring_idle();
                pushed = true;
                for (int t0 = 0; t0 < tile.ntok; t0 += 8) {
                    float r[HALVES][8];
                    const int n = min(8, tile.ntok - t0);
                    read8(t0, n, r);
                    float *out = smem_out + buf * 8 * OUT;
                    if (nsplit > 1) {
                        push(tile, t0, n, r);
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (j >= n) break;
                        if (UP) {
                            out[j * OUT + mine] = gated(r[0][j], r[HALVES - 1][j]);
                        } else {
#pragma unroll
                            for (int h = 0; h < HALVES; ++h) out[j * ROWS + h * 128 + mine] = r[h][j];
                        }
                    }
                    named_bar_sync(1, 128);
                    write_out(tile, out, t0, n);
                    buf ^= 1;
                }
                release();
            }
        }
    epi_done:
        __syncwarp();
        if (nsplit > 1 && !pushed) ring_idle();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
    if (UP || nsplit == 1) return;
    // ---------------------------------------------------------------- sum over the cluster (one tile)
    if (first_tile < num_tiles) {
        const FewTile tile = get_tile(first_tile);
        const int rows = min(share, tile.ntok * ROW_GROUPS - rank * share);
        if (rows <= 0) return;   // (nobody writes here)
        if (threadIdx.x == 0) mbar_arrive_expect_tx(join_bar, nsplit * rows * COMP * 128);
        if (!mbar_wait_cluster_warp(join_bar, 0, ctl, DG_DEV_TIMEOUT)) {
            // A peer may still write here: leave with it (threads that have left count as arrived).
            cluster_arrive();
            cluster_wait();
            return;
        }
        for (int row = warp; row < rows; row += blockDim.x / 32) {
            float sum[COMP] = {}, o[4];
#pragma unroll 4
            for (int r = 0; r < nsplit; ++r)
#pragma unroll
                for (int c = 0; c < COMP; ++c) sum[c] += smem_out[((r * share + row) * COMP + c) * 32 + lane];
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = sum[c];
            const int at = rank * share + row;
            store(tile, at / ROW_GROUPS, tile.row0 + (at % ROW_GROUPS) * 128 + 4 * lane, o);
        }
    }
}

}  // namespace dg
