// Products of a few bf16 rows with FP4 or FP8 weights, and the two kernels of the MoE
// layer for few tokens, on the block-scaled tensor cores.
//
// The weights are the MMA's 128-row operand, straight from their packed form (TMA
// unpacks E2M1 to one code per byte of shared memory; their UE8M0 scales go to TMEM
// as they are), so no instruction touches a weight.  The activations are the narrow
// operand: each value x of a group of 32 along K is split into two E4M3 pieces
//     x = s (hi + lo / 16),  s = 2^(floor(log2 max|x|) - 7),
// which occupy two adjacent columns with the scales s and s/16.  hi holds 4 significant
// bits and lo the 4 that follow (with its sign, 9 bits in all), so a bf16 value is
// represented exactly down to 2^-13 of its group's largest, and to 2^-21 of the largest
// below that.  An FP32 value (the layer's inner activations) is rounded to 9 bits, half
// a bf16 unit.  Products and sums are FP32 in TMEM; the two columns are added at the end.
//
// With M = 128 weight rows an MMA of K = 32 takes as long as its 4 KB of weights take
// to be read from shared memory up to N = 64 columns (32 rows of activations), which is a
// third of the time they take from HBM: the weight stream is the bound.
//
// A CTA computes tiles of HALVES x 128 weight rows, over K-blocks of 128 K:
//   warp 0      producer: weights by TMA (a 3-D box that takes weight row 4l + c to
//               operand row 32c + l, so that 128 consecutive scale words are already in
//               the order in which tcgen05.cp takes them to TMEM), scales by bulk copy.
//   warp 1      TMEM owner, MMA issuer.
//   warps 2..5  epilogue, one TMEM lane quadrant each.
//   warps 6..9  the narrow operand, K-blocks in turn.
// Many tiles: the CTAs are persistent and take tiles in turn, the ring of K-blocks running
// on across them.  Few tiles: one tile per cluster, K split over its CTAs, which add
// their FP32 partial results in rank order through distributed shared memory: no
// workspace, no atomics, a fixed order.
//
// Modes, by where the pieces come from:
//   kGemv   the warps split the activations themselves.
//   kGemvPre  dg_few_split_kernel has split them once, into rows [2m][K] of codes and
//           per K-block a 512-byte block of scale words in tcgen05.cp order: TMA loads.
//   kUp     the gate and up rows of one expert (HALVES = 2) for up to `cap` of the tokens
//           routed to it, whose split rows are gathered.  The epilogue is w silu(g) u (w
//           the routing weight), split again into pieces.
//   kDown   K runs over all active experts; a column belongs to one token throughout
//           and is zero for the experts that the token does not use, so the sum over a
//           token's experts is the accumulation itself.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dg_internal.h"
#include "ptx.cuh"

namespace dg {

enum FewMode : int { kGemv = 0, kGemvPre = 1, kUp = 2, kDown = 3 };

struct FewArgs {
    const uint16_t *x;      // kGemv: bf16 activations
    int64_t ldx;
    const uint8_t *codes;   // kUp, kDown: split rows, codes [2 rows][K] (row 2r hi, 2r + 1 lo)
    const uint32_t *scales; // their scale words [K / 128][2 rows]; kGemvPre: [K / 128][128] in tcgen05.cp order
    uint8_t *out_codes;     // kUp: the same of its output, rows = t * topk
    uint8_t *out_scales;
    const uint32_t *sf;     // packed scale words of the weights
    int64_t sf_expert;      // words per expert
    int sf_ld;              // words per slice
    int rows;               // weight rows of one expert (kUp: 2 i)
    int tokens;             // rows of x
    int src_rows;           // kUp, kDown: rows of the split source (t, t * topk)
    int kblocks;            // K-blocks of one expert
    int cap;                // token columns of the operand (8, 16, 32 or 64); N = 2 cap
    int stages;
    int accs;               // accumulator sets (1 or 2)
    int tmem_cols;
    int row_tiles;          // tiles over the weight rows (kUp: of h's columns)
    int chunks;             // kUp: groups of cap tokens that an expert may have
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
};

struct FewConfig {
    static constexpr int kThreads = 320;
    static constexpr int kFirstEpi = 2, kFirstB = 6, kBWarps = 4;
    static constexpr int kAlign = 1024;
    static constexpr int kBarBytes = 512;
    static constexpr int kMaxStages = 24;
    static int stage_bytes(int halves, int cap) { return halves * 16384 + 2 * cap * 128 + halves * 512 + 512; }
    // two buffers of 8 tokens' FP32 results (split tiles leave theirs in the ring)
    static int out_bytes(int halves, int mode, int split) {
        return split > 1 ? 0 : 2 * 8 * (mode == kUp ? 128 : halves * 128) * 4;
    }
    static int table_bytes(int mode, int pairs) { return mode < kUp ? 0 : (256 + 24 * pairs + 15) / 16 * 16; }
    static int smem_bytes(int halves, int cap, int stages, int mode, int pairs, int split) {
        return kAlign + stages * stage_bytes(halves, cap) + out_bytes(halves, mode, split) + kBarBytes +
               table_bytes(mode, pairs);
    }
};

// Four scaled values to their hi and lo pieces.
__device__ __forceinline__ void split4(float f0, float f1, float f2, float f3, uint32_t &hi, uint32_t &lo) {
    const uint32_t h01 = cvt_e4m3x2(f0, f1), h23 = cvt_e4m3x2(f2, f3);
    const uint32_t b01 = e4m3x2_to_f16x2(h01), b23 = e4m3x2_to_f16x2(h23);
    const float2 g01 = __half22float2(*reinterpret_cast<const __half2 *>(&b01));
    const float2 g23 = __half22float2(*reinterpret_cast<const __half2 *>(&b23));
    hi = h01 | (h23 << 16);
    lo = cvt_e4m3x2((f0 - g01.x) * 16.0f, (f1 - g01.y) * 16.0f) |
         (cvt_e4m3x2((f2 - g23.x) * 16.0f, (f3 - g23.y) * 16.0f) << 16);
}

// Biased exponent of a group's largest magnitude, kept where both scales are representable;
// 255 marks an infinity or a NaN in the group, whose scales become NaN.
__device__ __forceinline__ uint32_t hi_scale(uint32_t e8) { return e8 == 255u ? 255u : e8 - 7u; }
__device__ __forceinline__ uint32_t lo_scale(uint32_t e8) { return e8 == 255u ? 255u : e8 - 11u; }
__device__ __forceinline__ float inverse_scale(uint32_t e8) { return __uint_as_float((261u - e8) << 23); }

// Lane q16 of 16 holds values 8 q16 .. 8 q16 + 7 of one row's K-block (4 lanes to a group
// of 32): their pieces, and the group's exponent.
__device__ __forceinline__ uint32_t split_bf16(const uint4 &v, uint2 &hi, uint2 &lo) {
    const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    uint32_t m = max(m2 >> 16, m2 & 0xFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t e8 = max(m >> 7, 11u);
    const float inv = inverse_scale(e8);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16) * inv;
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * inv;
    }
    split4(f[0], f[1], f[2], f[3], hi.x, lo.x);
    split4(f[4], f[5], f[6], f[7], hi.y, lo.y);
    return e8;
}

// Position of operand row n's scale word in a 512-byte block (tcgen05.cp order).
__device__ __forceinline__ uint32_t sf_word(uint32_t n) { return (n & 31u) * 4u + (n >> 5); }

// Splits bf16 rows once for all CTAs that read them: 16 lanes per row and K-block.
__global__ void __launch_bounds__(256) dg_few_split_kernel(const uint16_t *x, int64_t ldx, int rows, int kblocks,
                                                           uint8_t *codes, uint32_t *scales, int cp_order) {
    grid_dependency_wait();
    grid_launch_dependents();   // after the wait: the next kernel may read what was there before this one
    const int unit = blockIdx.x * 16 + static_cast<int>(threadIdx.x >> 4);
    const int q16 = threadIdx.x & 15;
    const bool in = unit < rows * kblocks;
    const int kb = in ? unit / rows : 0, t = in ? unit % rows : 0;
    const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(x + t * ldx + kb * 128 + q16 * 8));
    uint2 hi, lo;
    const uint32_t e8 = split_bf16(v, hi, lo);
    if (!in) return;
    const int64_t k = static_cast<int64_t>(kblocks) * 128;
    uint8_t *at = codes + 2 * t * k + kb * 128 + q16 * 8;
    *reinterpret_cast<uint2 *>(at) = hi;
    *reinterpret_cast<uint2 *>(at + k) = lo;
    if ((q16 & 3) == 0) {
        const uint32_t n = 2 * t;
        uint8_t *s = reinterpret_cast<uint8_t *>(cp_order ? scales + kb * 128 + sf_word(n)
                                                          : scales + static_cast<int64_t>(kb) * 2 * rows + n) + (q16 >> 2);
        s[0] = static_cast<uint8_t>(hi_scale(e8));
        s[cp_order ? 16 : 4] = static_cast<uint8_t>(lo_scale(e8));
    }
}

// One tile of work, the same for every role of a CTA.
struct FewTile {
    int expert;     // kUp
    int row0;       // first weight row (kUp: column of h)
    int ntok;       // token columns
    int ent;        // kUp: first entry
    int begin;      // first K-block (kDown: over the active experts)
    int nblk;
};

template <bool FP4, int HALVES, int MODE>
__global__ void __launch_bounds__(FewConfig::kThreads, 2)
    dg_few_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const __grid_constant__ FewArgs p) {
    constexpr int ROWS = HALVES * 128;
    constexpr int OUT = MODE == kUp ? 128 : ROWS;     // results per token and tile
    constexpr int NT = FewConfig::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int S = p.stages;
    const int ncols = 2 * p.cap;
    const int b_bytes = ncols * 128;
    uint8_t *smem_a = smem;
    uint8_t *smem_b = smem_a + S * HALVES * 16384;
    uint8_t *smem_sfa = smem_b + S * b_bytes;
    uint8_t *smem_sfb = smem_sfa + S * HALVES * 512;
    float *smem_out = reinterpret_cast<float *>(smem_sfb + S * 512);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem_out + (cluster_nctarank() > 1 ? 0 : 2 * 8 * OUT));
    uint64_t *full_bar = bars;              // [S] weights and scales landed, pieces written
    uint64_t *empty_bar = bars + S;         // [S] the slot's MMAs are done
    uint64_t *tfull_bar = bars + 2 * S;     // [2] accumulators complete
    uint64_t *tempty_bar = tfull_bar + 2;   // [2] accumulators read
    uint64_t *drain_bar = tempty_bar + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *sh_active = reinterpret_cast<int *>(tmem_holder + 2);
    int *tab = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + FewConfig::kBarBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};
    const int rank = static_cast<int>(cluster_ctarank());
    const int nsplit = static_cast<int>(cluster_nctarank());
    const int first_tile = blockIdx.x / nsplit, tile_step = gridDim.x / nsplit;

    if (warp == 0) {
        for (int i = lane; i < 2 * S + 5; i += 32)
            mbar_init(bars + i, i < S ? 2 : i == 2 * S + 2 || i == 2 * S + 3 ? 4 : 1);
        if (lane == 0) {
            *abort_flag = 0;
            tma_prefetch_desc(&tm_w);
            if (MODE == kGemvPre) tma_prefetch_desc(&tm_x);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, p.tmem_cols);
        tmem_relinquish();
    }
    // The first kernel of a chain (kGemv; the split kernel before the others) waits for
    // what precedes it and only then lets the next one start.  So the later kernels of
    // the chain may read weights, ids and routing weights at once; only the warps that
    // read the preceding kernel's output wait for it.
    if constexpr (MODE == kGemv) grid_dependency_wait();
    grid_launch_dependents();

    // ---------------------------------------------------------------- routing tables
    const int pairs = MODE < kUp ? 0 : p.tokens * p.topk;
    uint32_t *tab_mask = reinterpret_cast<uint32_t *>(tab);   // [32] experts in use
    int *tab_pre = tab + 32;                                  // [32] experts in use before this word
    int *s_ids = tab + 64;                                    // [pairs] id of a token's first slot with it, or -1
    float *s_wsum = reinterpret_cast<float *>(s_ids + pairs); // [pairs] by entry: weight (of all the token's slots)
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(s_wsum + pairs);     // [active][2] tokens of each expert
    uint16_t *s_ent = reinterpret_cast<uint16_t *>(s_mask + 2 * pairs);  // [pairs] by entry: first slot (pair)
    uint16_t *s_off = s_ent + pairs;                          // [active] end of each expert's entries
    uint16_t *s_exp = s_off + pairs;                          // [active] expert
    int active = 1;
    if constexpr (MODE >= kUp) {
        if (warp == 0) tab_mask[lane] = 0u;
        __syncthreads();
        for (int q = threadIdx.x; q < pairs; q += NT) {
            int e = __ldcg(p.ids + q);
            if (e >= p.experts) {
                if (p.status) atomicOr(p.status, DG_DEV_BAD_GROUP);
                e = -1;
            }
            for (int r = q - q % p.topk; r < q && e >= 0; ++r)
                if (__ldcg(p.ids + r) == e) e = -1;
            s_ids[q] = e < 0 ? -1 : e;
            if (e >= 0) atomicOr(&tab_mask[e >> 5], 1u << (e & 31));
        }
        __syncthreads();
        if (warp == 0) {
            const int cnt = __popc(tab_mask[lane]);
            int inc = cnt;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, s);
                if (lane >= s) inc += v;
            }
            tab_pre[lane] = inc - cnt;
            if (lane == 31) *sh_active = inc;
            const int used = __shfl_sync(0xFFFFFFFFu, inc, 31);
            for (int a = lane; a < used; a += 32) {
                s_off[a] = 0;
                s_mask[2 * a] = s_mask[2 * a + 1] = 0u;
            }
            __syncwarp();
            // one warp counts, scans and fills, in slot order (the order is the same in every CTA)
            auto rank_of = [&](int e) {
                return e < 0 ? -1 - lane : tab_pre[e >> 5] + __popc(tab_mask[e >> 5] & ((1u << (e & 31)) - 1));
            };
            for (int q0 = 0; q0 < pairs; q0 += 32) {
                const int e = q0 + lane < pairs ? s_ids[q0 + lane] : -1;
                const int a = rank_of(e);
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, a);
                if (a >= 0 && (same >> lane) == 1u) {   // the last holder of this expert
                    s_off[a] += static_cast<uint16_t>(__popc(same));
                    s_exp[a] = static_cast<uint16_t>(e);
                }
                __syncwarp();
            }
            int run = 0;
            for (int a0 = 0; a0 < used; a0 += 32) {
                const int n = a0 + lane < used ? s_off[a0 + lane] : 0;
                int sum = n;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const int v = __shfl_up_sync(0xFFFFFFFFu, sum, s);
                    if (lane >= s) sum += v;
                }
                if (a0 + lane < used) s_off[a0 + lane] = static_cast<uint16_t>(run + sum - n);
                run += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
            __syncwarp();
            for (int q0 = 0; q0 < pairs; q0 += 32) {
                const int q = q0 + lane;
                const int e = q < pairs ? s_ids[q] : -1;
                const int a = rank_of(e);
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, a);
                if (a >= 0) {
                    const int at = s_off[a] + __popc(same & ((1u << lane) - 1));
                    const int token = q / p.topk;
                    s_ent[at] = static_cast<uint16_t>(q);
                    if constexpr (MODE == kUp) {
                        float w = 0.0f;
                        for (int r = q; r < (token + 1) * p.topk; ++r)
                            if (__ldcg(p.ids + r) == e) w += __ldcg(p.weights + r);
                        s_wsum[at] = w;
                    }
                    atomicOr(&s_mask[2 * a + (token >> 5)], 1u << (token & 31));
                }
                __syncwarp();
                if (a >= 0 && (same >> lane) == 1u) s_off[a] += static_cast<uint16_t>(__popc(same));
                __syncwarp();
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    if constexpr (MODE >= kUp) active = *sh_active;
    const int total = MODE == kDown ? active * p.kblocks : p.kblocks;     // K-blocks of a tile
    const int num_tiles = MODE == kUp ? active * p.row_tiles * p.chunks : p.row_tiles;
    const int k_begin = static_cast<int>(static_cast<int64_t>(total) * rank / nsplit);
    const int k_count = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / nsplit) - k_begin;

    // Tile w: kUp's go expert by expert, an expert's groups of tokens next to each other
    // (they read the same weights).  False: no tokens.
    auto get_tile = [&](int w, FewTile &t) -> bool {
        t.begin = k_begin;
        t.nblk = k_count;
        t.ent = 0;
        if constexpr (MODE == kUp) {
            const int chunk = w % p.chunks, at = w / p.chunks;
            const int a = at / p.row_tiles;
            const int first = (a ? s_off[a - 1] : 0) + chunk * p.cap;
            t.row0 = (at - a * p.row_tiles) * 128;
            t.expert = s_exp[a];
            t.ent = first;
            t.ntok = min(static_cast<int>(s_off[a]) - first, p.cap);
            return t.ntok > 0;
        } else {
            t.expert = 0;
            t.row0 = w * ROWS;
            t.ntok = p.tokens;
            return true;
        }
    };
    // Four results of one token at weight rows n .. n + 3 (kUp: a warp holds the token's 128).
    auto store = [&](const FewTile &tile, int t, int n, float (&o)[4]) {
        if constexpr (MODE == kUp) {
            const float w = s_wsum[tile.ent + t];
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                o[c] *= w;
                m = max(m, __float_as_uint(o[c]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));   // a group of 32
            const uint32_t e8 = max(m >> 23, 11u);
            const float inv = inverse_scale(e8);
            uint32_t hi, lo;
            split4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv, hi, lo);
            const int64_t row = 2 * static_cast<int64_t>(s_ent[tile.ent + t]);
            *reinterpret_cast<uint32_t *>(p.out_codes + row * p.inner + n) = hi;
            *reinterpret_cast<uint32_t *>(p.out_codes + (row + 1) * p.inner + n) = lo;
            if ((lane & 7) == 0) {
                uint8_t *sf = p.out_scales + ((tile.row0 >> 7) * 2 * static_cast<int64_t>(pairs) + row) * 4 + (lane >> 3);
                sf[0] = static_cast<uint8_t>(hi_scale(e8));
                sf[4] = static_cast<uint8_t>(lo_scale(e8));
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
    auto gated = [](float g, float u) { return g / (1.0f + expf(-g)) * u; };

    FewTile tile;
    float *part = reinterpret_cast<float *>(smem_a);   // nsplit > 1: [ntok][ROWS], in operand row order

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int slot = 0;
        uint32_t phase = 0;
        uint32_t issued = 0;
        bool drop = (p.debug_flags & DG_DEBUG_DROP_ONE_LOAD) && blockIdx.x == 0;
        for (int w = first_tile; w < num_tiles; w += tile_step) {
            if (!get_tile(w, tile)) continue;
            int a = 0, kb = tile.begin;
            if (MODE == kDown) { a = kb / p.kblocks; kb -= a * p.kblocks; }
            for (int i = 0; i < tile.nblk; ++i) {
                if (!mbar_wait_warp(&empty_bar[slot], phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto producer_done;
                if (drop) drop = false;   // diagnostic: this slot never fills
                else issued |= 1u << slot;
                if ((issued >> slot & 1u) && elect_one()) {
                    const int e = MODE == kDown ? s_exp[a] : tile.expert;
                    const int slice = FP4 ? kb : kb >> 2;
                    const uint32_t *sf = p.sf + e * p.sf_expert + static_cast<int64_t>(slice) * p.sf_ld;
                    uint32_t sf_bytes[HALVES];
                    uint32_t bytes = HALVES * (FP4 ? 8192 : 16384);
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const int left = MODE == kUp ? 128 : p.sf_ld - (tile.row0 + h * 128);
                        sf_bytes[h] = left >= 128 ? 512u : left > 0 ? 4u * static_cast<uint32_t>(left) : 0u;
                        bytes += sf_bytes[h];
                    }
                    mbar_arrive_expect_tx(&full_bar[slot], bytes);
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const int r = MODE == kUp ? h * p.inner + tile.row0 : tile.row0 + h * 128;
                        // (a half past the last row reads zeros or the next expert's rows; unused)
                        const int64_t r4 = (static_cast<int64_t>(e) * p.rows + r) >> 2;
                        tma_load_3d(smem_a + (slot * HALVES + h) * 16384, &tm_w, &full_bar[slot], kb * 128,
                                    static_cast<int32_t>(r4), 0);
                        if (sf_bytes[h])
                            bulk_load(smem_sfa + (slot * HALVES + h) * 512, sf + r, sf_bytes[h], &full_bar[slot]);
                    }
                }
                __syncwarp();
                if (++kb == p.kblocks && MODE == kDown) { kb = 0; ++a; }
                if (++slot == S) { slot = 0; phase ^= 1; }
            }
        }
    producer_done:
        // Normally every load has landed once the MMAs are done.  After a wait that ran
        // out, never leave with loads in flight: give them the time limit once more.
        named_bar_sync(2, 64);   // the MMA warp is done with its waits
        if (lane == 0 && *abort_flag) {
            const uint64_t t0 = global_timer_ns();
            for (int s = 0; s < S; ++s)
                while ((issued & (1u << s)) && global_timer_ns() - t0 < ctl.timeout_ns &&
                       !mbar_try_wait(smem_u32(&full_bar[s]), s < slot ? phase : phase ^ 1)) {}
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        int slot = 0, acc = 0, g = 0;
        uint32_t phase = 0, acc_phase = 0;
        const uint64_t a_base = make_desc_kmajor_sw128(smem_u32(smem_a));
        const uint64_t b_base = make_desc_kmajor_sw128(smem_u32(smem_b));
        const uint32_t sf_tmem = tmem_base + p.accs * HALVES * ncols;   // two slots of 4 HALVES + 4 columns
        for (int w = first_tile; w < num_tiles; w += tile_step) {
            if (!get_tile(w, tile)) continue;
            if (!mbar_wait_warp(&tempty_bar[acc], acc_phase ^ 1, ctl, DG_DEV_TIMEOUT)) goto mma_done;
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + acc * HALVES * ncols;
            // columns in use: the tokens', rounded up to the MMA's step of 16
            const int n_used = MODE == kUp ? (2 * tile.ntok + 15) / 16 * 16 : ncols;
            const uint32_t idesc = make_idesc_mxf8(128, n_used, 0, 0) | (FP4 ? 5u << 7 : 0u);   // A: E2M1 or E4M3
            int kb = MODE == kDown ? tile.begin % p.kblocks : tile.begin;
            for (int i = 0; i < tile.nblk; ++i, ++g) {
                if (!mbar_wait_warp(&full_bar[slot], phase, ctl, DG_DEV_TIMEOUT)) goto mma_done;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint32_t sf = sf_tmem + (g & 1) * (4 * HALVES + 4);
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
                        tc_cp_32x128b_warpx4(sf + 4 * h,
                                             make_desc_sf_32x128b(smem_u32(smem_sfa + (slot * HALVES + h) * 512)));
                    tc_cp_32x128b_warpx4(sf + 4 * HALVES, make_desc_sf_32x128b(smem_u32(smem_sfb + slot * 512)));
                    const uint64_t b_desc = b_base + static_cast<uint64_t>(slot * (b_bytes >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // scale byte: the activations' and FP4 weights' k-th 32 K, FP8 weights' 128-K block
                        const uint32_t id = idesc | (static_cast<uint32_t>(k) << 4) |
                                            (static_cast<uint32_t>(FP4 ? k : kb & 3) << 29);
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            tc_mma_mxf8(d_tmem + h * ncols,
                                        a_base + static_cast<uint64_t>((slot * HALVES + h) * 1024 + 2 * k),
                                        b_desc + 2 * k, id, sf + 4 * h, sf + 4 * HALVES, (i | k) != 0);
                    }
                    tc_commit(&empty_bar[slot]);
                }
                __syncwarp();
                if (++kb == p.kblocks) kb = 0;
                if (++slot == S) { slot = 0; phase ^= 1; }
            }
            if (elect_one()) tc_commit(&tfull_bar[acc]);
            __syncwarp();
            if (++acc == p.accs) { acc = 0; acc_phase ^= 1; }
        }
    mma_done:
        // TMEM is not freed before every MMA has finished
        if (elect_one()) {
            tc_commit(drain_bar);
            mbar_wait_drain(drain_bar, 0, ctl);
        }
        __syncwarp();
        named_bar_sync(2, 64);
    } else if (warp >= FewConfig::kFirstB) {
        // ------------------------------------------------------------ the narrow operand
        // The warps take the K-blocks in turn, at most as many warps as ring slots: a
        // wait for the MMAs of block g - S tests one parity bit, which is unambiguous only
        // if block g - 2S is known to be done; a warp's previous block g - teams implies that
        // up to block g - teams - S.
        const int teams = S < FewConfig::kBWarps ? S : FewConfig::kBWarps;
        const int bw = warp - FewConfig::kFirstB;
        const int q16 = lane & 15, sub = lane >> 4;   // two tokens at a time, 16 lanes each
        if constexpr (MODE != kGemv) grid_dependency_wait();
        int g = 0;   // K-blocks of the tiles before
        for (int w = first_tile; w < num_tiles && bw < teams; w += tile_step) {
            if (!get_tile(w, tile)) continue;
            for (int i = (bw + teams - g % teams) % teams; i < tile.nblk; i += teams) {
                const int slot = (g + i) % S;
                if (!mbar_wait_warp(&empty_bar[slot], (((g + i) / S) & 1) ^ 1, ctl, DG_DEV_TIMEOUT)) goto b_done;
                uint8_t *tile_b = smem_b + slot * b_bytes;
                uint8_t *tile_sf = smem_sfb + slot * 512;
                int kb = tile.begin + i, a = 0;
                if (MODE == kDown) { a = kb / p.kblocks; kb -= a * p.kblocks; }
                if constexpr (MODE == kGemvPre) {
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full_bar[slot], b_bytes + 512);
                        tma_load_2d(tile_b, &tm_x, &full_bar[slot], kb * 128, 0);
                        bulk_load(tile_sf, p.scales + kb * 128, 512, &full_bar[slot]);
                    }
                    __syncwarp();
                    continue;
                } else if constexpr (MODE == kGemv) {
                    for (int t0 = 0; t0 < tile.ntok; t0 += 8) {
                        uint4 v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int t = t0 + 2 * u + sub;
                            v[u] = make_uint4(0u, 0u, 0u, 0u);
                            if (t < tile.ntok)
                                v[u] = __ldcg(reinterpret_cast<const uint4 *>(p.x + t * p.ldx + kb * 128 + q16 * 8));
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (t0 + 2 * u >= tile.ntok) break;
                            const int t = t0 + 2 * u + sub;
                            uint2 hi, lo;
                            const uint32_t e8 = split_bf16(v[u], hi, lo);
                            if (t >= tile.ntok) continue;
                            // columns 2t and 2t + 1 (rows of 128 bytes, 128-byte swizzle)
                            const uint32_t n = 2 * t;
                            const uint32_t off = (q16 & 1) * 8;
                            *reinterpret_cast<uint2 *>(tile_b + n * 128 + (((q16 >> 1) ^ (n & 7)) << 4) + off) = hi;
                            *reinterpret_cast<uint2 *>(tile_b + (n + 1) * 128 + (((q16 >> 1) ^ ((n + 1) & 7)) << 4) +
                                                       off) = lo;
                            if ((q16 & 3) == 0) {
                                uint8_t *s = tile_sf + sf_word(n) * 4 + (q16 >> 2);
                                s[0] = static_cast<uint8_t>(hi_scale(e8));
                                s[16] = static_cast<uint8_t>(lo_scale(e8));
                            }
                        }
                        __syncwarp();
                    }
                } else {
                    int begin = tile.ent, end = tile.ent + tile.ntok;
                    if constexpr (MODE == kDown) {
                        // columns of tokens that do not use this expert are zero, codes and scales
                        for (int t = sub; t < p.cap; t += 2) {
                            if (s_mask[2 * a + (t >> 5)] >> (t & 31) & 1u) continue;
                            reinterpret_cast<uint4 *>(tile_b + t * 256)[q16] = make_uint4(0u, 0u, 0u, 0u);
                            if (q16 < 2) reinterpret_cast<uint32_t *>(tile_sf)[sf_word(2 * t + q16)] = 0u;
                        }
                        __syncwarp();
                        begin = a ? s_off[a - 1] : 0;
                        end = s_off[a];
                    }
                    const int64_t k = static_cast<int64_t>(p.kblocks) * 128;
                    const uint8_t *src = p.codes + (q16 >> 3) * k + kb * 128 + (q16 & 7) * 16;
                    const uint32_t *src_sf = p.scales + static_cast<int64_t>(kb) * 2 * p.src_rows + (q16 & 1);
                    for (int t0 = begin; t0 < end; t0 += 8) {
                        uint4 v[4];
                        uint32_t sf[4];
                        int col[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int t = t0 + 2 * u + sub;
                            if (t < end) {
                                const int pair = s_ent[t];
                                const int token = pair / p.topk;
                                const int row = MODE == kUp ? token : pair;
                                col[u] = MODE == kUp ? t - begin : token;
                                v[u] = __ldcg(reinterpret_cast<const uint4 *>(src + 2 * row * k));
                                sf[u] = __ldcg(src_sf + 2 * row);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (t0 + 2 * u + sub < end) {
                                const uint32_t n = 2 * col[u] + (q16 >> 3);
                                *reinterpret_cast<uint4 *>(tile_b + n * 128 + (((q16 & 7) ^ (n & 7)) << 4)) = v[u];
                                if (q16 < 2) reinterpret_cast<uint32_t *>(tile_sf)[sf_word(2 * col[u] + q16)] = sf[u];
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full_bar[slot]);
            }
            g += tile.nblk;
        }
    b_done:
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const uint32_t quad = warp & 3;
        const int id = threadIdx.x - 32 * FewConfig::kFirstEpi;   // 0..127
        int acc = 0, buf = 0;
        uint32_t acc_phase = 0;
        if constexpr (MODE != kGemv) grid_dependency_wait();       // C, and memory that the output may share
        for (int w = first_tile; w < num_tiles; w += tile_step) {
            if (!get_tile(w, tile)) continue;
            // the four warps go on or give up together
            const bool ok = mbar_wait_warp(&tfull_bar[acc], acc_phase, ctl, DG_DEV_TIMEOUT);
            if (!named_bar_and(1, 128, ok)) break;
            tc_fence_after_sync();
            for (int t0 = 0; t0 < tile.ntok; t0 += 8) {
                uint32_t v[HALVES][16];
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[h][j] = 0u;
                    if (tile.nblk > 0)
                        tmem_ld_32x32b_x16(tmem_base + ((quad * 32) << 16) + (acc * HALVES + h) * ncols + 2 * t0, v[h]);
                }
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < HALVES; ++h) reg_fence16(v[h]);
                if (t0 + 8 >= tile.ntok) {   // the accumulators are read
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty_bar[acc]);
                }
                float *out = nsplit > 1 ? part + t0 * ROWS : smem_out + buf * 8 * OUT;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (t0 + j >= tile.ntok) break;
                    float r[HALVES];
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
                        r[h] = __uint_as_float(v[h][2 * j]) + __uint_as_float(v[h][2 * j + 1]);
                    if (MODE == kUp && nsplit == 1) {
                        out[j * OUT + quad * 32 + lane] = gated(r[0], r[HALVES - 1]);
                    } else {
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) out[j * ROWS + h * 128 + quad * 32 + lane] = r[h];
                    }
                }
                if (nsplit > 1) continue;
                named_bar_sync(1, 128);
                const int n = min(8, tile.ntok - t0) * (OUT / 4);
                for (int q = id; q < n; q += 128) {
                    const int t = q / (OUT / 4), l = q % (OUT / 4);
                    float o[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[c] = out[t * OUT + (l >> 5) * 128 + 32 * c + (l & 31)];
                    store(tile, t0 + t, tile.row0 + 4 * l, o);
                }
                buf ^= 1;
            }
            if (++acc == p.accs) { acc = 0; acc_phase ^= 1; }
        }
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
    if (nsplit == 1) return;
    // ---------------------------------------------------------------- sum over the cluster (one tile)
    cluster_sync();
    if (first_tile < num_tiles && get_tile(first_tile, tile)) {
        const uint32_t part0 = smem_u32(smem_a);
        auto sum = [&](int idx) {
            float s = 0.0f;
            for (int r = 0; r < nsplit; ++r) s += ld_shared_cluster_f32(mapa_shared(part0 + 4u * idx, r));
            return s;
        };
        for (int q = rank * NT + threadIdx.x; q < tile.ntok * (OUT / 4); q += nsplit * NT) {
            const int t = q / (OUT / 4), l = q % (OUT / 4);
            const int base = t * ROWS + (l >> 5) * 128 + (l & 31);
            float o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                o[c] = sum(base + 32 * c);
                if constexpr (MODE == kUp) o[c] = gated(o[c], sum(base + 128 + 32 * c));
            }
            store(tile, t, tile.row0 + 4 * l, o);
        }
    }
    __syncwarp();
    cluster_sync();   // peers may still read this CTA's partial results
}

}  // namespace dg
