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
// A CTA computes HALVES x 128 weight rows over a range of K-blocks (128 K each):
//   warp 0      producer: weights by TMA (a 3-D box that takes weight row 4l + c to
//               operand row 32c + l, so that 128 consecutive scale words are already in
//               the order in which tcgen05.cp takes them to TMEM), scales by bulk copy.
//   warp 1      TMEM owner, MMA issuer.
//   warps 2..9  the narrow operand, then the epilogue.
// K is split over the CTAs of a cluster, which add their FP32 partial results in rank
// order through distributed shared memory: no workspace, no atomics, a fixed order.
//
// Modes, by where the pieces come from:
//   kGemv   teams of warps split the activations themselves, a K-block at a time.
//   kGemvPre  dg_few_split_kernel has split them once, into rows [2m][K] of codes and
//           per K-block a 512-byte block of scale words in tcgen05.cp order; one warp
//           loads them by TMA.
//   kUp     the gate and up rows of one expert (HALVES = 2) for the tokens routed to it;
//           teams of warps gather the tokens' split rows.  The epilogue is w silu(g) u (w
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
    int tmem_cols;
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
    static constexpr int kConvWarps = 8;
    static constexpr int kFirstConv = 2;
    static constexpr int kAlign = 1024;
    static constexpr int kBarBytes = 512;
    static constexpr int kMaxStages = 24;
    static int stage_bytes(int halves, int cap) { return halves * 16384 + 2 * cap * 128 + halves * 512 + 512; }
    static int table_bytes(int mode, int pairs) { return mode < kUp ? 0 : (256 + 24 * pairs + 15) / 16 * 16; }
    static int smem_bytes(int halves, int cap, int stages, int mode, int pairs) {
        return kAlign + stages * stage_bytes(halves, cap) + kBarBytes + table_bytes(mode, pairs);
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

template <bool FP4, int HALVES, int MODE>
__global__ void __launch_bounds__(FewConfig::kThreads, 2)
    dg_few_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const __grid_constant__ FewArgs p) {
    constexpr int ROWS = HALVES * 128;
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
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem_sfb + S * 512);
    uint64_t *full_bar = bars;              // [S] weights and scales landed (transactions), pieces written by the team
    uint64_t *empty_bar = bars + S;         // [S] the slot's MMAs are done
    uint64_t *tfull_bar = bars + 2 * S;     // the accumulators are complete
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(tfull_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *tab = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + FewConfig::kBarBytes);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, p.status, p.timeout_ns};
    const int rank = static_cast<int>(cluster_ctarank());
    const int nsplit = static_cast<int>(cluster_nctarank());
    const int tile = blockIdx.x / nsplit;
    // Converter teams: at most one per ring slot.  A team's wait for the MMAs of block
    // i - S tests one parity bit, which is unambiguous only if block i - 2S is known to be
    // done; the team's previous block i - teams implies that up to block i - teams - S.
    const int teams = S < FewConfig::kConvWarps ? S : FewConfig::kConvWarps;
    const int team_size = MODE == kGemvPre ? 1 : FewConfig::kConvWarps / teams;

    if (warp == 0) {
        for (int i = lane; i < 2 * S + 1; i += 32) mbar_init(bars + i, i < S ? 1 + team_size : 1);
        if (lane == 0) {
            *abort_flag = 0;
            tma_prefetch_desc(&tm_w);
            if (MODE == kGemvPre) tma_prefetch_desc(&tm_x);
        }
        fence_mbar_init();
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
    float *s_wsum = reinterpret_cast<float *>(s_ids + pairs); // kUp: by entry, the weight (of all the token's slots)
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(s_wsum + pairs);  // kDown [active][2] tokens of each expert
    uint16_t *s_ent = reinterpret_cast<uint16_t *>(s_mask + 2 * pairs);   // kUp: pairs of this CTA; kDown: by entry
    uint16_t *s_off = s_ent + pairs;                          // kDown [active] end of each expert's entries
    uint16_t *s_exp = s_off + pairs;                          // kDown [active] expert
    __shared__ int sh_active, sh_expert, sh_count;
    int ntok = p.tokens;
    int expert = 0;
    int active = 1;
    if constexpr (MODE >= kUp) {
        if (warp == 0) tab_mask[lane] = 0u;
        if (threadIdx.x == 0) { sh_count = 0; sh_expert = 0; }
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
            const uint32_t word = tab_mask[lane];
            const int cnt = __popc(word);
            int inc = cnt;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, s);
                if (lane >= s) inc += v;
            }
            const int before = inc - cnt;
            tab_pre[lane] = before;
            if (lane == 31) sh_active = inc;
            if constexpr (MODE == kUp) {
                const int a = blockIdx.y;
                if (a >= before && a < inc) {
                    uint32_t w = word;
                    for (int s = before; s < a; ++s) w &= w - 1;
                    sh_expert = lane * 32 + __ffs(w) - 1;
                }
            }
        }
        __syncthreads();
        active = sh_active;
        if constexpr (MODE == kUp) {
            // the tokens of this CTA's expert, in order, from the blockIdx.z-th group of cap
            expert = sh_expert;
            if (warp == 0 && static_cast<int>(blockIdx.y) < active) {
                const int first = blockIdx.z * p.cap;
                int n = 0;
                for (int q0 = 0; q0 < pairs; q0 += 32) {
                    const bool hit = q0 + lane < pairs && s_ids[q0 + lane] == expert;
                    const uint32_t m = __ballot_sync(0xFFFFFFFFu, hit);
                    const int at = n + __popc(m & ((1u << lane) - 1)) - first;
                    if (hit && at >= 0 && at < p.cap) {
                        const int q = q0 + lane, token0 = q - q % p.topk;
                        float w = 0.0f;
                        for (int r = q; r < token0 + p.topk; ++r)
                            if (__ldcg(p.ids + r) == expert) w += __ldcg(p.weights + r);
                        s_ent[at] = static_cast<uint16_t>(q);
                        s_wsum[at] = w;
                    }
                    n += __popc(m);
                }
                if (lane == 0) sh_count = max(0, min(n - first, p.cap));
            }
            __syncthreads();
            ntok = sh_count;
            if (ntok == 0) {   // no such expert or group of tokens; the same for the whole cluster
                grid_dependency_wait();
                return;
            }
        } else {
            // entries of all active experts, grouped by expert
            for (int a = threadIdx.x; a < active; a += NT) {
                s_off[a] = 0;
                s_mask[2 * a] = s_mask[2 * a + 1] = 0u;
            }
            __syncthreads();
            if (warp == 0) {
                // few hundred slots: one warp counts, scans and fills in slot order
                for (int q0 = 0; q0 < pairs; q0 += 32) {
                    const int e = q0 + lane < pairs ? s_ids[q0 + lane] : -1;
                    const int a = e < 0 ? -1 - lane : tab_pre[e >> 5] + __popc(tab_mask[e >> 5] & ((1u << (e & 31)) - 1));
                    const uint32_t same = __match_any_sync(0xFFFFFFFFu, a);
                    if (a >= 0 && (same >> lane) == 1u) {   // the last holder of this expert
                        s_off[a] += static_cast<uint16_t>(__popc(same));
                        s_exp[a] = static_cast<uint16_t>(e);
                    }
                    __syncwarp();
                }
                int run = 0;
                for (int a0 = 0; a0 < active; a0 += 32) {
                    const int cnt = a0 + lane < active ? s_off[a0 + lane] : 0;
                    int inc = cnt;
#pragma unroll
                    for (int s = 1; s < 32; s <<= 1) {
                        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, s);
                        if (lane >= s) inc += v;
                    }
                    if (a0 + lane < active) s_off[a0 + lane] = static_cast<uint16_t>(run + inc - cnt);
                    run += __shfl_sync(0xFFFFFFFFu, inc, 31);
                    __syncwarp();
                }
                for (int q0 = 0; q0 < pairs; q0 += 32) {
                    const int q = q0 + lane;
                    const int e = q < pairs ? s_ids[q] : -1;
                    const int a = e < 0 ? -1 - lane : tab_pre[e >> 5] + __popc(tab_mask[e >> 5] & ((1u << (e & 31)) - 1));
                    const uint32_t same = __match_any_sync(0xFFFFFFFFu, a);
                    if (a >= 0) {
                        const int at = s_off[a] + __popc(same & ((1u << lane) - 1));
                        s_ent[at] = static_cast<uint16_t>(q);
                        atomicOr(&s_mask[2 * a + (q / p.topk >> 5)], 1u << (q / p.topk & 31));
                    }
                    __syncwarp();
                    if (a >= 0 && (same >> lane) == 1u) s_off[a] += static_cast<uint16_t>(__popc(same));
                    __syncwarp();
                }
            }
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;

    // this CTA's K-blocks
    const int total = MODE == kDown ? active * p.kblocks : p.kblocks;
    const int k_begin = static_cast<int>(static_cast<int64_t>(total) * rank / nsplit);
    const int nblk = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / nsplit) - k_begin;
    const int row0 = tile * (MODE == kUp ? 128 : ROWS);   // first weight row (kUp: of the gate half)

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int slot = 0;
        uint32_t phase = 0;
        uint32_t issued = 0;
        bool drop = (p.debug_flags & DG_DEBUG_DROP_ONE_LOAD) && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
        int a = MODE == kDown && total > 0 ? k_begin / p.kblocks : 0;
        int kb = MODE == kDown && total > 0 ? k_begin - a * p.kblocks : k_begin;
        for (int i = 0; i < nblk; ++i) {
            if (!mbar_wait_warp(&empty_bar[slot], phase ^ 1, ctl, DG_DEV_TIMEOUT)) break;
            if (drop) drop = false;   // diagnostic: this slot never fills
            else issued |= 1u << slot;
            if ((issued >> slot & 1u) && elect_one()) {
                const int e = MODE == kDown ? s_exp[a] : expert;
                const int slice = FP4 ? kb : kb >> 2;
                const uint32_t *sf = p.sf + e * p.sf_expert + static_cast<int64_t>(slice) * p.sf_ld;
                uint32_t sf_bytes[HALVES];
                uint32_t bytes = HALVES * (FP4 ? 8192 : 16384);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const int left = MODE == kUp ? 128 : p.sf_ld - (row0 + h * 128);
                    sf_bytes[h] = left >= 128 ? 512u : left > 0 ? 4u * static_cast<uint32_t>(left) : 0u;
                    bytes += sf_bytes[h];
                }
                mbar_arrive_expect_tx(&full_bar[slot], bytes);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    const int r = MODE == kUp ? h * p.inner + row0 : row0 + h * 128;
                    // (a half past the last row reads zeros)
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
        int slot = 0;
        uint32_t phase = 0;
        const uint64_t a_base = make_desc_kmajor_sw128(smem_u32(smem_a));
        const uint64_t b_base = make_desc_kmajor_sw128(smem_u32(smem_b));
        const uint32_t sf_tmem = tmem_base + HALVES * ncols;   // two slots of 4 HALVES + 4 columns
        // columns in use: the tokens', rounded up to the MMA's step of 16
        const int n_used = MODE == kUp ? (2 * ntok + 15) / 16 * 16 : ncols;
        const uint32_t idesc = make_idesc_mxf8(128, n_used, 0, 0) | (FP4 ? 5u << 7 : 0u);
        int kb = MODE == kDown && total > 0 ? k_begin % p.kblocks : k_begin;
        for (int i = 0; i < nblk; ++i) {
            if (!mbar_wait_warp(&full_bar[slot], phase, ctl, DG_DEV_TIMEOUT)) break;
            tc_fence_after_sync();
            if (elect_one()) {
                const uint32_t sf = sf_tmem + (i & 1) * (4 * HALVES + 4);
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
                        tc_mma_mxf8(tmem_base + h * ncols,
                                    a_base + static_cast<uint64_t>((slot * HALVES + h) * 1024 + 2 * k), b_desc + 2 * k,
                                    id, sf + 4 * h, sf + 4 * HALVES, (i | k) != 0);
                }
                tc_commit(&empty_bar[slot]);
            }
            __syncwarp();
            if (++kb == p.kblocks) kb = 0;
            if (++slot == S) { slot = 0; phase ^= 1; }
        }
        // the accumulators are complete; TMEM is not freed before every MMA has finished
        if (elect_one()) {
            tc_commit(tfull_bar);
            mbar_wait_drain(tfull_bar, 0, ctl);
        }
        __syncwarp();
        named_bar_sync(2, 64);
    } else {
        // ------------------------------------------------------------ the narrow operand
        const int cw = warp - FewConfig::kFirstConv;
        if constexpr (MODE != kGemv) grid_dependency_wait();
        if constexpr (MODE == kGemvPre) {
            for (int i = cw; i < nblk && cw == 0; ++i) {
                const int slot = i % S;
                if (!mbar_wait_warp(&empty_bar[slot], ((i / S) & 1) ^ 1, ctl, DG_DEV_TIMEOUT)) break;
                if (elect_one()) {
                    const int kb = k_begin + i;
                    mbar_arrive_expect_tx(&full_bar[slot], b_bytes + 512);
                    tma_load_2d(smem_b + slot * b_bytes, &tm_x, &full_bar[slot], kb * 128, 0);
                    bulk_load(smem_sfb + slot * 512, p.scales + kb * 128, 512, &full_bar[slot]);
                }
                __syncwarp();
            }
        } else {
            const int team = cw / team_size, member = cw % team_size;
            const int q16 = lane & 15, sub = lane >> 4;   // two tokens at a time, 16 lanes each
            int a = 0, kb = k_begin + team;
            if (MODE == kDown && total > 0) { a = kb / p.kblocks; kb -= a * p.kblocks; }
            for (int i = team < teams ? team : nblk; i < nblk; i += teams) {
                const int slot = i % S;
                if (!mbar_wait_warp(&empty_bar[slot], ((i / S) & 1) ^ 1, ctl, DG_DEV_TIMEOUT)) break;
                uint8_t *tile_b = smem_b + slot * b_bytes;
                uint8_t *tile_sf = smem_sfb + slot * 512;
                if constexpr (MODE == kGemv) {
                    for (int t0 = 8 * member; t0 < ntok; t0 += 8 * team_size) {
                        uint4 v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int t = t0 + 2 * u + sub;
                            v[u] = make_uint4(0u, 0u, 0u, 0u);
                            if (t < ntok)
                                v[u] = __ldcg(reinterpret_cast<const uint4 *>(p.x + t * p.ldx + kb * 128 + q16 * 8));
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (t0 + 2 * u >= ntok) break;
                            const int t = t0 + 2 * u + sub;
                            uint2 hi, lo;
                            const uint32_t e8 = split_bf16(v[u], hi, lo);
                            if (t >= ntok) continue;
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
                    }
                } else {
                    int begin = 0, end = ntok;
                    if constexpr (MODE == kDown) {
                        // columns of tokens that do not use this expert are zero, codes and scales
                        for (int t = 2 * member + sub; t < p.cap; t += 2 * team_size) {
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
                    for (int t0 = begin + 8 * member; t0 < end; t0 += 8 * team_size) {
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
                                col[u] = MODE == kUp ? t : token;
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
                kb += teams;
                if constexpr (MODE == kDown)
                    while (kb >= p.kblocks) { kb -= p.kblocks; ++a; }
            }
        }

        // ------------------------------------------------------------ accumulators -> shared memory
        // (the ring is free: every load has landed and every MMA has read its slot)
        float *part = reinterpret_cast<float *>(smem_a);      // [ntok][ROWS], in operand row order
        const uint32_t quad = warp & 3;
        const int group = cw >> 2;
        if (nblk > 0) {
            __all_sync(0xFFFFFFFFu, mbar_wait(tfull_bar, 0, ctl, DG_DEV_TIMEOUT));
            tc_fence_after_sync();
        }
        const int half = HALVES == 2 ? group : 0;
        for (int c = HALVES == 2 ? 0 : group; c * 8 < ntok; c += HALVES == 2 ? 1 : 2) {
            uint32_t v[16] = {};
            if (nblk > 0) {
                tmem_ld_32x32b_x16(tmem_base + ((quad * 32) << 16) + half * ncols + c * 16, v);
                tmem_ld_wait();
                reg_fence16(v);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c * 8 + j < ntok)
                    part[(c * 8 + j) * ROWS + half * 128 + quad * 32 + lane] =
                        __uint_as_float(v[2 * j]) + __uint_as_float(v[2 * j + 1]);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
    // (the grid must not end before the one it depends on, whoever else waited)
    if constexpr (MODE != kGemv) grid_dependency_wait();
    if (nsplit > 1) cluster_sync();
    // ---------------------------------------------------------------- sum over the cluster, output
    const uint32_t part0 = smem_u32(smem_a);
    auto load = [&](int idx) {
        float s = 0.0f;
        if (nsplit == 1) return reinterpret_cast<const float *>(smem_a)[idx];
        for (int r = 0; r < nsplit; ++r) s += ld_shared_cluster_f32(mapa_shared(part0 + 4u * idx, r));
        return s;
    };
    constexpr int QUADS = MODE == kUp ? 32 : HALVES * 32;     // groups of 4 outputs per token
    for (int q = rank * NT + threadIdx.x; q < ntok * QUADS; q += nsplit * NT) {
        const int t = q / QUADS, l = q % QUADS;
        const int base = t * ROWS + (l >> 5) * 128 + (l & 31);
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = load(base + 32 * c);
        const int n = row0 + 4 * l;
        if constexpr (MODE == kUp) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float u = load(base + 128 + 32 * c);
                o[c] = o[c] / (1.0f + expf(-o[c])) * u;
            }
            // a warp holds one token's 128 values; 8 lanes a group of 32
            const float w = s_wsum[t];
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                o[c] *= w;
                m = max(m, __float_as_uint(o[c]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
            const uint32_t e8 = max(m >> 23, 11u);
            const float inv = inverse_scale(e8);
            uint32_t hi, lo;
            split4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv, hi, lo);
            const int64_t row = 2 * static_cast<int64_t>(s_ent[t]);
            *reinterpret_cast<uint32_t *>(p.out_codes + row * p.inner + n) = hi;
            *reinterpret_cast<uint32_t *>(p.out_codes + (row + 1) * p.inner + n) = lo;
            if ((lane & 7) == 0) {
                uint8_t *sf = p.out_scales + ((row0 >> 7) * 2 * static_cast<int64_t>(pairs) + row) * 4 + (lane >> 3);
                sf[0] = static_cast<uint8_t>(hi_scale(e8));
                sf[4] = static_cast<uint8_t>(lo_scale(e8));
            }
        } else if (n < p.rows) {
            if (p.f32) {
                if (p.c) {
                    const float4 c = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.c) + t * p.ldc + n));
                    o[0] += c.x; o[1] += c.y; o[2] += c.z; o[3] += c.w;
                }
                *reinterpret_cast<float4 *>(static_cast<float *>(p.d) + t * p.ldd + n) =
                    make_float4(o[0], o[1], o[2], o[3]);
            } else {
                if (p.c) {
                    const uint2 c = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.c) + t * p.ldc + n));
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
    }
    if (nsplit > 1) cluster_sync();   // peers may still read this CTA's partial results
}

}  // namespace dg
