// Host side of the feed-forward training entry points of include/dg.h: the gated
// block and its backward pass, the FP8 quantiser, Newton-Schulz orthogonalisation.
// Validation order as in api.cu: sizes, pointers, alignment, then the device.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "dg_internal.h"

namespace dg {
namespace {

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align4(int64_t x) { return (x + 3) / 4 * 4; }

// 2-D tensor map; true if it was encoded.
bool encode(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t dim0, uint64_t dim1,
            uint64_t stride_bytes, uint32_t box0, uint32_t box1, CUtensorMapSwizzle swizzle,
            CUtensorMapL2promotion promo) {
    TensorMapEncodeFn fn = host_encode();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {dim0, dim1};
    const cuuint64_t strides[1] = {stride_bytes};
    const cuuint32_t box[2] = {box0, box1};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// FP8 operand: boxes of 128 bytes x `rows`, 128-byte swizzle.
bool encode_fp8(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint64_t ld, uint32_t rows) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, inner, outer, ld, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// bf16 output: boxes of 32 columns x 32 rows, 64-byte swizzle.
bool encode_out(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, int64_t ld) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, cols, rows, static_cast<uint64_t>(ld) * 2, 32, 32,
                  CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// Co-resident clusters of a gated kernel on the current device, in num_sms SMs (the cluster's size
// is that of the kernel: a pair, or forward the pairs that share a group of 128 columns).
int gated_clusters(int bn, bool backward, int num_sms) {
    static std::mutex mu;
    static int cache[64][2][3];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int &v = cache[dev][backward ? 1 : 0][bn == 256 ? 0 : bn == 128 ? 1 : 2];
    if (v == 0) v = bs2_max_active_pairs(bn, false, 256, false, backward ? (kLayGatedBwd | 2) : kLayGated);
    const int cluster = backward ? 2 : 512 / bn;
    return v * cluster > num_sms ? num_sms / cluster : v;
}

// Columns of the tiles.  Forward: 256 (128 gate, 128 up), or where that leaves pairs without a tile 128 or
// 64, with 2 or 4 pairs to a group of 128 columns of h; a K-block takes what its loads take, 16 KB
// of rows and 64 bytes a column at about 55 bytes a cycle (64 columns: 0.62 of 256).  7 rows, inner 1408,
// k 2048: 8.8 us with 64 columns, 9.8 with 256; 128 rows, inner 2048, k 7168: 18.0 against 20.8 (14.0
// with ring slots of two K-blocks).  Backward: a K-block of B is loaded whole whatever the tile's
// columns, so 128 only where all its tiles run at once, with half the epilogue (515 rows, inner 1360,
// k 2048: 12.2 us against 16.8 with 256; 1 row, inner 2048, k 7168: 18.3 against 23.8).
// units: grouped, the least there can be, as if every block of 128 rows had another of its expert beside it (where
// the experts' rows lie is known to the device alone).  Experts of a single block make up to twice as many, and a
// call with tiles chosen for one wave then takes two.
int gated_block_n(bool backward, int64_t units, int inner, int num_sms) {
    if (backward) {
        const int64_t tiles = units * cdiv(inner, 128);
        return tiles <= gated_clusters(128, true, num_sms) ? 128 : 256;
    }
    int best = 256;
    double least = 0.0;
    const int64_t groups = units * cdiv(inner, kGran);
    for (int bn : {256, 128, 64}) {
        const int clusters = gated_clusters(bn, false, num_sms);
        if (clusters <= 0) continue;
        const double t = static_cast<double>(cdiv(groups, clusters)) * (16384 + 64 * bn);
        if (bn == 256 || t < 0.97 * least) {
            best = bn;
            least = t;
        }
    }
    return best;
}

struct GatedArgs {
    const void *a;       // x, or dy
    int64_t lda;
    const void *sfa;
    const void *b;       // W1 [groups][2 inner][ldb], or W2 [groups][k][ldb]
    int64_t ldb;
    const void *sfb;
    const int32_t *layout;   // grouped: expert of each row; nullptr: dense
    void *gu;
    int64_t ldgu;
    void *h;
    int64_t ldh;
    void *hq;
    int64_t ldhq;
    void *sfh;
    void *dgu;
    int64_t lddgu;
    int m, inner, k, groups;
    bool grouped, backward;
    int32_t *status;
    void *stream;
};

bool bad_out(const void *p, int64_t ld) { return !aligned(p, 16) || ld % 8 != 0; }

dg_status gated(const GatedArgs &g) {
    const int m = g.m, inner = g.inner, k = g.k;
    if (m < 0 || inner < 0 || k < 0 || g.groups < 1) return DG_ERR_INVALID_ARG;
    if (g.grouped && m % kBlockM != 0) return DG_ERR_LAYOUT;
    if (m == 0 || inner == 0) return DG_OK;
    if (k == 0 || m > kMaxFewSize || inner > kMaxFewSize / 2 || k > kMaxFewSize) return DG_ERR_UNSUPPORTED;
    const int64_t units = cdiv(m, 2 * kBlockM);
    const int64_t max_units = g.grouped ? m / kBlockM : units;
    const int64_t b_rows = static_cast<int64_t>(g.groups) * (g.backward ? k : 2 * inner);
    if (max_units * cdiv(inner, 128) > INT32_MAX / 8 || b_rows > INT32_MAX) return DG_ERR_UNSUPPORTED;
    if (g.grouped && (units > kMaxPairPrefix || g.groups >= 32768)) return DG_ERR_UNSUPPORTED;
    // pointers
    if (!g.a || !g.b || !g.sfa || !g.sfb || (g.grouped && !g.layout)) return DG_ERR_INVALID_ARG;
    if (g.backward ? (!g.gu || !g.dgu) : (!g.h == !g.hq || (g.hq && !g.sfh))) return DG_ERR_INVALID_ARG;
    if (g.lda < k || g.ldb < (g.backward ? inner : k) || (g.gu && g.ldgu < 2 * static_cast<int64_t>(inner)) ||
        (g.h && g.ldh < inner) || (g.hq && g.ldhq < inner) ||
        (g.dgu && g.lddgu < 2 * static_cast<int64_t>(inner)))
        return DG_ERR_INVALID_ARG;
    // alignment: 16-byte rows; whole 16-column chunks of the inner width; whole K-blocks where
    // an expert's rows of B follow another's along K
    if (!aligned(g.a, 16) || !aligned(g.b, 16) || !aligned(g.sfa, 16) || !aligned(g.sfb, 16) || !aligned(g.layout, 4))
        return DG_ERR_ALIGNMENT;
    if (inner % 16 != 0 || k % 16 != 0 || (g.backward && g.grouped && k % kBlockK != 0) || g.lda % 16 != 0 ||
        g.ldb % 16 != 0)
        return DG_ERR_ALIGNMENT;
    if ((g.gu && bad_out(g.gu, g.ldgu)) || (g.h && bad_out(g.h, g.ldh)) || (g.dgu && bad_out(g.dgu, g.lddgu)) ||
        (g.hq && (!aligned(g.hq, 16) || g.ldhq % 16 != 0 || !aligned(g.sfh, 16))))
        return DG_ERR_ALIGNMENT;
    int sms = 0;
    dg_status st = host_check_device(&sms, nullptr);
    if (st != DG_OK) return st;

    GemmParams p;
    std::memset(&p, 0, sizeof(p));
    p.mode = g.grouped ? kModeContiguous : kModeDense;
    p.rows = m;
    p.n = inner;
    p.k = k;
    p.num_groups = g.groups;
    p.grouped_layout = g.layout;
    p.status = g.status;
    p.layout = g.backward ? (kLayGatedBwd | 2) : kLayGated;
    p.num_m_blocks = static_cast<int>(units);
    const int bn = gated_block_n(g.backward, units, inner, sms);
    p.num_n_blocks = static_cast<int>(cdiv(inner, g.backward ? bn : kGran));
    p.num_k_blocks = static_cast<int>(cdiv(k, kBlockK));
    p.group_m = 8;
    p.timeout_ns = host_timeout_ns();
    p.debug_flags = host_take_debug_flags();
    const int64_t psf_k = cdiv(p.num_k_blocks, 4);
    p.sfa_words = static_cast<const uint32_t *>(g.sfa);
    p.sfb_words = static_cast<const uint32_t *>(g.sfb);
    p.sfa_ld = static_cast<int>(align4(m));
    p.sfb_ld = static_cast<int>(align4(g.backward ? inner : 2 * static_cast<int64_t>(inner)));
    p.sfa_slices = static_cast<int>(psf_k);
    p.sfb_slices = static_cast<int>(psf_k * g.groups);
    p.gu = static_cast<uint16_t *>(g.gu);
    p.ldgu = g.ldgu;
    TensorMaps maps;
    p.few_rows = !g.grouped && m <= kBlockM ? (m + 7) / 8 * 8 : 0;
    bool ok = encode_fp8(&maps.a, g.a, k, m, g.lda, p.few_rows > 0 ? p.few_rows : kBlockM);
    if (g.backward) {
        p.d = static_cast<uint16_t *>(g.dgu);
        p.ldd = g.lddgu;
        p.h = static_cast<uint16_t *>(g.h);
        p.ldh = g.ldh;
        ok &= encode_fp8(&maps.b, g.b, inner, b_rows, g.ldb, kBlockK);
        maps.d = maps.c = maps.a;   // not used
    } else {
        p.d = static_cast<uint16_t *>(g.h);
        p.ldd = g.ldh;
        p.hq = static_cast<uint8_t *>(g.hq);
        p.ldhq = g.ldhq;
        p.sfh = static_cast<uint8_t *>(g.sfh);
        p.sfh_ld = static_cast<int>(align4(m));
        ok &= encode_fp8(&maps.b, g.b, k, b_rows, g.ldb, static_cast<uint32_t>(bn / 2));
        if (g.h) ok &= encode_out(&maps.d, g.h, inner, m, g.ldh);
        if (g.gu) ok &= encode_out(&maps.c, g.gu, 2 * static_cast<uint64_t>(inner), m, g.ldgu);
        if (!g.h) maps.d = g.gu ? maps.c : maps.a;   // not used
        if (!g.gu) maps.c = maps.d;
    }
    maps.b2 = maps.b;   // not used
    if (!ok) return DG_ERR_CUDA;
    KernelInfo info;
    const int clusters = gated_clusters(bn, g.backward, sms), cluster = g.backward ? 2 : 512 / bn;
    if (clusters <= 0 || !get_bs2_kernel_info(bn, false, 256, &info, false, p.layout)) return DG_ERR_UNSUPPORTED;
    const int64_t tiles = max_units * p.num_n_blocks;
    const int grid = cluster * static_cast<int>(tiles < clusters ? tiles : clusters);
    host_set_last_config(256, bn, info.stages, grid, 2, 1);
    if ((p.debug_flags & DG_DEBUG_PRINT_CONFIGS) || std::getenv("DG_PRINT_CONFIGS"))
        std::fprintf(stderr, "[dg] gated %s rows=%d inner=%d k=%d -> BLOCK_M=256 BLOCK_N=%d stages=%d smem=%d grid=%d\n",
                     g.backward ? "backward" : "forward", m, inner, k, bn, info.stages, info.smem_bytes, grid);
    const cudaError_t e = launch_bs2_gemm(bn, 256, maps, p, grid, static_cast<cudaStream_t>(g.stream));
    return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

bool ns_unsupported(int batch, int rows, int cols) {
    return batch > 4096 || rows > kMaxNsSide || cols > kMaxNsSide || static_cast<int64_t>(rows) * cols > kMaxNsElements;
}

// The products' grid counters, 32 bits whose differences are signed, count both CTAs of each finished
// tile: at most 6 a step and tile of 256 x 64, the narrowest.
bool ns_too_many_tiles(int batch, int rows, int cols, int steps) {
    const int64_t lo = rows < cols ? rows : cols, hi = rows < cols ? cols : rows;
    return 6ll * steps * batch * cdiv(lo, 256) * cdiv(hi, 64) > INT32_MAX;
}

bool bad_values(const void *x, int64_t ldx, int fmt) {
    return !aligned(x, 16) || ldx % (fmt == DG_VALUES_BF16 ? 8 : 4) != 0;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_fp8_gated_gemm_nt(const void *a, int64_t lda, const void *sfa, const void *b, int64_t ldb, const void *sfb,
                               void *gu, int64_t ldgu, void *h, int64_t ldh, void *hq, int64_t ldhq, void *sfh, int m,
                               int inner, int k, int32_t *status_dev, void *stream) {
    GatedArgs g = {};
    g.a = a; g.lda = lda; g.sfa = sfa; g.b = b; g.ldb = ldb; g.sfb = sfb;
    g.gu = gu; g.ldgu = ldgu; g.h = h; g.ldh = ldh; g.hq = hq; g.ldhq = ldhq; g.sfh = sfh;
    g.m = m; g.inner = inner; g.k = k; g.groups = 1;
    g.status = status_dev; g.stream = stream;
    return gated(g);
}

dg_status dg_m_grouped_fp8_gated_gemm_nt_contiguous(const void *a, int64_t lda, const void *sfa, const void *b,
                                                    int64_t ldb, const void *sfb, void *gu, int64_t ldgu, void *h,
                                                    int64_t ldh, void *hq, int64_t ldhq, void *sfh,
                                                    const int32_t *grouped_layout, int m_total, int inner, int k,
                                                    int num_groups, int32_t *status_dev, void *stream) {
    GatedArgs g = {};
    g.a = a; g.lda = lda; g.sfa = sfa; g.b = b; g.ldb = ldb; g.sfb = sfb;
    g.gu = gu; g.ldgu = ldgu; g.h = h; g.ldh = ldh; g.hq = hq; g.ldhq = ldhq; g.sfh = sfh;
    g.layout = grouped_layout; g.grouped = true;
    g.m = m_total; g.inner = inner; g.k = k; g.groups = num_groups;
    g.status = status_dev; g.stream = stream;
    return gated(g);
}

dg_status dg_fp8_gated_gemm_nn_backward(const void *dy, int64_t lddy, const void *sfdy, const void *w2, int64_t ldw2,
                                        const void *sfw2, const void *gu, int64_t ldgu, void *dgu, int64_t lddgu,
                                        void *h, int64_t ldh, int m, int inner, int k, int32_t *status_dev,
                                        void *stream) {
    GatedArgs g = {};
    g.a = dy; g.lda = lddy; g.sfa = sfdy; g.b = w2; g.ldb = ldw2; g.sfb = sfw2;
    g.gu = const_cast<void *>(gu); g.ldgu = ldgu; g.dgu = dgu; g.lddgu = lddgu; g.h = h; g.ldh = ldh;
    g.m = m; g.inner = inner; g.k = k; g.groups = 1; g.backward = true;
    g.status = status_dev; g.stream = stream;
    return gated(g);
}

dg_status dg_m_grouped_fp8_gated_gemm_nn_backward_contiguous(const void *dy, int64_t lddy, const void *sfdy,
                                                             const void *w2, int64_t ldw2, const void *sfw2,
                                                             const void *gu, int64_t ldgu, void *dgu, int64_t lddgu,
                                                             void *h, int64_t ldh, const int32_t *grouped_layout,
                                                             int m_total, int inner, int k, int num_groups,
                                                             int32_t *status_dev, void *stream) {
    GatedArgs g = {};
    g.a = dy; g.lda = lddy; g.sfa = sfdy; g.b = w2; g.ldb = ldw2; g.sfb = sfw2;
    g.gu = const_cast<void *>(gu); g.ldgu = ldgu; g.dgu = dgu; g.lddgu = lddgu; g.h = h; g.ldh = ldh;
    g.layout = grouped_layout; g.grouped = true; g.backward = true;
    g.m = m_total; g.inner = inner; g.k = k; g.groups = num_groups;
    g.status = status_dev; g.stream = stream;
    return gated(g);
}

dg_status dg_quantize_fp8(const void *x, int x_fmt, int64_t ldx, void *q, int64_t ldq, void *sf, void *qk, int64_t ldqk,
                          void *sfk, int rows, int cols, const int *ks, int num_groups, void *stream) {
    if (rows < 0 || cols < 0 || num_groups < 0) return DG_ERR_INVALID_ARG;
    if (x_fmt != DG_VALUES_F32 && x_fmt != DG_VALUES_BF16) return DG_ERR_INVALID_ARG;
    KGroupRows t;
    t.num_groups = 0;
    if (ks != nullptr) {
        if (host_k_grouped_rows(ks, num_groups, &t) < 0) return DG_ERR_INVALID_ARG;
        if (cols % 4 != 0 || static_cast<int64_t>(t.srow[num_groups]) * kBlockK != rows) return DG_ERR_LAYOUT;
    }
    if (rows == 0 || cols == 0) return DG_OK;
    if (rows > kMaxQuantSize || cols > kMaxQuantSize) return DG_ERR_UNSUPPORTED;
    if (!x || (!q && !qk) || (ks && !qk) || (q && !sf) || (qk && !sfk)) return DG_ERR_INVALID_ARG;
    if (ldx < cols || (q && ldq < cols) || (qk && ldqk < cols)) return DG_ERR_INVALID_ARG;
    if (bad_values(x, ldx, x_fmt) || (q && (!aligned(q, 16) || ldq % 16 != 0 || !aligned(sf, 16))) ||
        (qk && (!aligned(qk, 16) || ldqk % 16 != 0 || !aligned(sfk, 16))))
        return DG_ERR_ALIGNMENT;
    int sms = 0;
    dg_status st = host_check_device(&sms, nullptr);
    if (st != DG_OK) return st;
    QuantParams p = {};
    p.x = x;
    p.ldx = ldx;
    p.rows = rows;
    p.cols = cols;
    p.q = static_cast<uint8_t *>(q);
    p.ldq = ldq;
    p.sf = static_cast<uint8_t *>(sf);
    p.sf_ld = static_cast<int>(align4(rows));
    p.qk = static_cast<uint8_t *>(qk);
    p.ldqk = ldqk;
    p.sfk = static_cast<uint8_t *>(sfk);
    p.sfk_ld = static_cast<int>(align4(cols));
    const cudaError_t e = launch_quantize(p, t, 1, (q ? 1 : 0) | (qk ? 2 : 0), x_fmt == DG_VALUES_BF16, sms,
                                          static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

dg_status dg_quantize_fp8_blocks(const void *x, int x_fmt, int64_t ldx, int64_t x_batch, void *q, int64_t ldq,
                                 int64_t q_batch, void *sf, void *sft, int batch, int rows, int cols, void *stream) {
    if (batch < 0 || rows < 0 || cols < 0) return DG_ERR_INVALID_ARG;
    if (x_fmt != DG_VALUES_F32 && x_fmt != DG_VALUES_BF16) return DG_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || cols == 0) return DG_OK;
    if (rows > kMaxQuantSize || cols > kMaxQuantSize || batch > 65535) return DG_ERR_UNSUPPORTED;
    if (!x || !q || (!sf && !sft)) return DG_ERR_INVALID_ARG;
    if (ldx < cols || ldq < cols || x_batch < 0) return DG_ERR_INVALID_ARG;
    if (batch > 1 && q_batch < (rows - 1) * ldq + cols) return DG_ERR_INVALID_ARG;   // (the matrices' codes are apart)
    if (batch > 1 && (x_batch % (x_fmt == DG_VALUES_BF16 ? 8 : 4) != 0 || q_batch % 16 != 0)) return DG_ERR_ALIGNMENT;
    if (bad_values(x, ldx, x_fmt) || !aligned(q, 16) || ldq % 16 != 0 || !aligned(sf, 16) || !aligned(sft, 16))
        return DG_ERR_ALIGNMENT;
    int sms = 0;
    dg_status st = host_check_device(&sms, nullptr);
    if (st != DG_OK) return st;
    QuantParams p = {};
    KGroupRows t;
    t.num_groups = 0;
    p.x = x;
    p.ldx = ldx;
    p.x_batch = x_batch;
    p.q_batch = q_batch;
    p.rows = rows;
    p.cols = cols;
    p.q = static_cast<uint8_t *>(q);
    p.ldq = ldq;
    p.sf = static_cast<uint8_t *>(sf);
    p.sf_ld = static_cast<int>(align4(rows));
    p.sfk = static_cast<uint8_t *>(sft);
    p.sfk_ld = static_cast<int>(align4(cols));
    const cudaError_t e = launch_quantize(p, t, batch, 4, x_fmt == DG_VALUES_BF16, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

int64_t dg_newton_schulz_workspace_bytes(int batch, int rows, int cols) {
    if (batch < 0 || rows < 0 || cols < 0 || ns_unsupported(batch, rows, cols)) return -1;
    return ns_workspace_bytes(batch, rows, cols);
}

dg_status dg_newton_schulz(const void *g, int g_fmt, int64_t ldg, int64_t g_batch, void *out, int64_t ldo,
                           int64_t out_batch, int batch, int rows, int cols, int steps, float a, float b, float c,
                           float eps, void *workspace, int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    if (batch < 0 || rows < 0 || cols < 0 || steps < 1 || !(eps >= 0.0f)) return DG_ERR_INVALID_ARG;
    if (g_fmt != DG_VALUES_F32 && g_fmt != DG_VALUES_BF16) return DG_ERR_INVALID_ARG;
    if (batch == 0 || rows == 0 || cols == 0) return DG_OK;
    if (ns_unsupported(batch, rows, cols) || steps > kMaxNsSteps || ns_too_many_tiles(batch, rows, cols, steps))
        return DG_ERR_UNSUPPORTED;
    if (!g || !out || !workspace || ldg < cols || ldo < cols) return DG_ERR_INVALID_ARG;
    if (g_batch < 0 || (batch > 1 && out_batch < (rows - 1) * ldo + cols)) return DG_ERR_INVALID_ARG;
    if (workspace_bytes < ns_workspace_bytes(batch, rows, cols)) return DG_ERR_INVALID_ARG;
    if (!aligned(g, g_fmt == DG_VALUES_F32 ? 4 : 2) || !aligned(out, 2) || !aligned(workspace, 128)) return DG_ERR_ALIGNMENT;
    int sms = 0;
    dg_status st = host_check_device(&sms, nullptr);
    if (st != DG_OK) return st;
    if (sms < 2) return DG_ERR_UNSUPPORTED;   // (CTA pairs)
    NsParams p = {};
    p.g = g;
    p.ldg = ldg;
    p.g_batch = g_batch;
    p.out = static_cast<uint16_t *>(out);
    p.ldo = ldo;
    p.out_batch = out_batch;
    p.batch = batch;
    p.rows = rows;
    p.cols = cols;
    p.ca = a;
    p.cb = b;
    p.cc = c;
    p.eps = eps;
    p.workspace = workspace;
    p.status = status_dev;
    p.timeout_ns = host_timeout_ns();
    p.debug_flags = host_take_debug_flags();
    NsConfig v;
    const cudaError_t e = launch_newton_schulz(p, steps, g_fmt == DG_VALUES_BF16, sms, static_cast<cudaStream_t>(stream),
                                               &v);
    if (e != cudaSuccess) return DG_ERR_CUDA;
    host_set_last_config(256, v.bn_update, v.stages, v.grid, 6, v.launches);
    if ((p.debug_flags & DG_DEBUG_PRINT_CONFIGS) || std::getenv("DG_PRINT_CONFIGS"))
        std::fprintf(stderr,
                     "[dg] newton-schulz batch=%d rows=%d cols=%d -> BLOCK_M=256 BLOCK_N=%d (symmetric) %d (update) "
                     "groups=%d+%d stages=%d grid=%d\n",
                     batch, rows, cols, v.bn_sym, v.bn_update, v.group0, batch - v.group0, v.stages, v.grid);
    return DG_OK;
}

}  // extern "C"
