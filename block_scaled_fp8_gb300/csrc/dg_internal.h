// Internal declarations shared by the host API and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg.h"  // include/ is on the include path

namespace dg {

constexpr int kBlockM = 128;   // rows per tile (one UMMA M=128, TMEM lanes)
constexpr int kBlockK = 128;   // K per pipeline stage (= scale granularity)
constexpr int kGran = 128;     // scale granularity along K (and N for FP32 B scales)
constexpr int kMaxGroupsMasked = 1024;
// Grouped layouts on CTA pairs: at most this many m-pairs (contiguous) or experts (masked).
constexpr int kMaxPairPrefix = 512;
// Experts of the PSUM contiguous layout (8-bit ids in the pair kernel's unit info).
constexpr int kMaxPsumGroups = 255;

enum GemmMode : int { kModeDense = 0, kModeContiguous = 1, kModeMasked = 2, kModeKGrouped = 3 };

// Runtime parameters of one GEMM launch (passed by value).
struct GemmParams {
    int mode;
    int rows;            // dense: M; contiguous: M_total; masked: max_m (rows per expert)
    int n, k;
    int num_m_blocks;    // blocks of 128 rows (dense/contiguous: over all rows; masked: per expert, max)
    int num_n_blocks;
    int num_k_blocks;
    int num_groups;
    int group_m;         // tile-order group size along M (L2 reuse)
    const int32_t *grouped_layout;  // contiguous: expert id per row
    const int32_t *psum;            // contiguous with PSUM offsets instead: [num_groups]
    const int32_t *masked_m;        // masked
    const int32_t *ks;              // K-grouped: rows of K per group [num_groups], multiples of 128
    int group_rows;                 // K-grouped: M, the rows of each group's D
    const uint16_t *c;   // dense: bf16 C or nullptr
    int64_t ldc;
    uint16_t *d;         // bf16 D (used for direct stores)
    float *d_f32;        // FP32 D (FP32-output GEMMs; then c_f32 is the FP32 C or null)
    const float *c_f32;
    int64_t ldd;
    int32_t *status;
    uint64_t timeout_ns;
    uint32_t debug_flags;
    int ab_3d;           // A/B tensor maps are the 3-D K-blocked views: one load per ring slot
    int c_v8;            // bf16 C rows are 32-byte aligned (base and ldc): 16 columns in one load
    int c_in_place;      // FP32 C is D itself (same pointer and stride): D is accumulated into at L2
    int c_tma;           // bf16 C goes through shared memory by TMA (dense pair GEMMs, 16-byte aligned rows)
    int layout;          // operand layouts: bit 0 A MN-major ([K][M]), bit 1 B MN-major ([K][N]),
                         // bit 2 B FP4 (E2M1, one scale per 32 K)
    // packed UE8M0 scale words, [slices][ld] int32 with ld = align4(mn); the
    // block-scaled kernels' scale warps read them with cp.async
    const uint32_t *sfa_words;
    const uint32_t *sfb_words;
    int sfa_ld, sfb_ld;
    int sfa_slices, sfb_slices;
    // FP32-promotion kernel only
    const float *sfa_f32;   // [rows][sf_k]
    const float *sfb_f32;   // [ceil(n/128)][sf_k]
    int sf_k;
};

struct TensorMaps {
    CUtensorMap a, b, d;
    CUtensorMap b2;   // pair tiles wider than 256 columns: the second MMA's rows of B
    CUtensorMap c;    // the pair kernel's bf16 C boxes (C tile in shared memory)
};

// Per-instantiation launch information.
struct KernelInfo {
    int block_n;
    int stages;
    int smem_bytes;
    int threads;
    int group_kb;   // K-blocks per ring slot (the depth of a 3-D A/B load)
    int num_acc;    // TMEM accumulators (1: the next tile's MMAs wait for the epilogue's reads)
};

// Block-scaled (UE8M0) tcgen05 kernel family: returns false if block_n is not
// compiled in.
bool get_bs_kernel_info(int block_n, bool with_c, KernelInfo *info);
cudaError_t launch_bs_gemm(int block_n, const TensorMaps &maps, const GemmParams &p, int grid,
                           cudaStream_t stream);

// CTA-pair (cta_group::2) block-scaled kernel family (the instantiations are
// listed in gemm_bs2_list.h).  mp = rows of a pair tile: 256 or 128; f32 picks
// the FP32-output (and FP32-C) epilogue; launch_bs2_gemm takes C and f32 from p.
bool get_bs2_kernel_info(int block_n, bool with_c, int mp, KernelInfo *info, bool f32 = false, int lay = 0);
cudaError_t launch_bs2_gemm(int block_n, int mp, const TensorMaps &maps, const GemmParams &p, int grid,
                            cudaStream_t stream);
int bs2_max_active_pairs(int block_n, bool with_c, int mp, bool f32 = false, int lay = 0);

// FP32-scale promotion kernel family.
bool get_promote_kernel_info(int block_n, KernelInfo *info);
cudaError_t launch_promote_gemm(int block_n, const TensorMaps &maps, const GemmParams &p, int grid,
                                cudaStream_t stream);

// Scale-factor transform.
// Scale rows of the K-grouped layout, per group: srow[e] = first 128-K block
// (FP32 scale row), prow[e] = first packed row; entries 0..num_groups.
struct KGroupRows {
    int num_groups;
    int srow[kMaxPsumGroups + 2];
    int prow[kMaxPsumGroups + 2];
};
cudaError_t launch_transform_sf_k_grouped(const float *sf, int mn, const KGroupRows &t, int packed_rows,
                                          void *out, int32_t *status, cudaStream_t stream);
cudaError_t launch_transform_sf(const float *sf, int batch, int mn_rows, int sf_k, int gran_mn,
                                int mn, int out_fmt, void *out, int32_t *status,
                                cudaStream_t stream);

// Host state and helpers of api.cu that the few-row entry points (api_few.cu) share.
typedef CUresult (*TensorMapEncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                      const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                      CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                      CUtensorMapFloatOOBfill);
dg_status host_check_device(int *num_sms, bool *limited);   // limited: dg_set_num_sms leaves some out
TensorMapEncodeFn host_encode();
uint64_t host_timeout_ns();
uint32_t host_take_debug_flags();   // clears DG_DEBUG_DROP_ONE_LOAD
void host_set_last_config(int block_m, int block_n, int stages, int grid, int kind, int launches);
cudaError_t launch_fill_d(const void *c, int64_t ldc, void *d, int64_t ldd, int m, int n, bool f32, int num_sms,
                          cudaStream_t stream);

// ---- few-row products, top-k routing and the MoE layer for few tokens

constexpr int kMaxFewRows = 64;         // rows of a few-row product, tokens of a MoE layer call
constexpr int kMaxFewSize = 0x7FFFFFFF - 255;   // n and k of a product, tokens to route: rounded up to tiles they fit an int
constexpr int kMaxLayerTopk = 16;
constexpr int kMaxLayerExperts = 1024;
constexpr int kMaxLayerWidth = 1 << 24;
constexpr int kMaxRouteExperts = 1024;
constexpr int kMaxRouteTopk = 32;

// One few-row product D = C + A @ B^T, bf16 A, FP4 or FP8 B with packed UE8M0 scales.
struct FewParams {
    const uint16_t *a;      // bf16 [m][lda]
    int64_t lda;
    const uint8_t *b;       // codes, row n at b + n * ldb bytes
    int64_t ldb;
    const uint32_t *sfb;    // [slices][align4(n)]
    const void *c;          // D's type, or nullptr
    int64_t ldc;
    void *d;
    int64_t ldd;
    int m, n, k;
    int fp4, f32;
    uint8_t *workspace;     // few_workspace_bytes(m, n, k)
    int32_t *status;
    uint64_t timeout_ns;
    uint32_t debug_flags;
};
int64_t few_workspace_bytes(int64_t m, int64_t n, int64_t k);
// max_occ (here and below): CTAs on an SM of the kernels that may have two
cudaError_t launch_few_gemv(const FewParams &p, int num_sms, int max_occ, cudaStream_t stream);

// The MoE layer for few tokens.
struct LayerParams {
    const uint16_t *x;      // bf16 [t][ldx]
    int64_t ldx;
    const int32_t *ids;     // [t][topk]
    const float *weights;   // [t][topk]
    const uint8_t *w1;      // [experts][2i][h] codes: gate rows, then up rows
    const uint32_t *sf1;
    const uint8_t *w2;      // [experts][h][i]
    const uint32_t *sf2;
    const uint16_t *c;      // bf16 [t][ldc] or nullptr
    int64_t ldc;
    uint16_t *y;            // bf16 [t][ldy]
    int64_t ldy;
    uint8_t *workspace;     // layer_workspace_bytes(t, topk, h, i, experts)
    int t, h, i, experts, topk;
    int fp4;
    int32_t *status;
    uint64_t timeout_ns;
    uint32_t debug_flags;
};
int64_t layer_workspace_bytes(int64_t t, int64_t topk, int64_t h, int64_t i, int64_t experts);
cudaError_t launch_moe_layer(const LayerParams &p, int num_sms, int max_occ, cudaStream_t stream);

struct RouteParams {
    const void *logits;
    int64_t ld;
    const float *bias;
    int32_t *ids;
    float *weights;
    int t, experts, topk;
    int bf16, sigmoid, renormalize;
    float scale;
    int vec, vec_bias;      // set by the launch: rows, the bias may be read 4 experts at a time
};
cudaError_t launch_moe_route(const RouteParams &p, cudaStream_t stream);

}  // namespace dg
