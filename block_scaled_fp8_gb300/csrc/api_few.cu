// Host side of the few-row entry points of include/dg.h: products of a few bf16
// rows with FP4 or FP8 weights, top-k routing, the MoE layer for few tokens.
// Validation order as in api.cu: sizes, pointers, alignment, then the device.
#include "dg_internal.h"

namespace dg {
namespace {

// The hardware lays CTAs out one to an SM before it puts a second on any, so a grid of two CTAs on each
// of `num_sms` SMs would take twice as many: where dg_set_num_sms leaves SMs out, an SM has one.
int max_occ(bool limited) { return limited ? 1 : 2; }

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

dg_status gemv(bool fp4, bool f32, const void *a, int64_t lda, const void *b, int64_t ldb, const void *sfb,
               const void *c, int64_t ldc, void *d, int64_t ldd, int m, int n, int k, void *workspace,
               int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    if (m < 0 || n < 0 || k < 0) return DG_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return DG_OK;
    if (m > kMaxFewRows || n > kMaxFewSize || k > kMaxFewSize) return DG_ERR_UNSUPPORTED;
    if (d == nullptr) return DG_ERR_INVALID_ARG;
    const int step = f32 ? 4 : 8;
    if (!aligned(d, 16) || ldd % step != 0 || n % 8 != 0) return DG_ERR_ALIGNMENT;
    if (ldd < n) return DG_ERR_INVALID_ARG;
    if (c != nullptr && (!aligned(c, 16) || ldc % step != 0)) return DG_ERR_ALIGNMENT;
    if (c != nullptr && ldc < n) return DG_ERR_INVALID_ARG;
    int sms = 0;
    if (k != 0) {
        if (a == nullptr || b == nullptr || sfb == nullptr) return DG_ERR_INVALID_ARG;
        if (k % kBlockK != 0) return DG_ERR_ALIGNMENT;
        if (!aligned(a, 16) || lda % 8 != 0 || !aligned(sfb, 16)) return DG_ERR_ALIGNMENT;
        const unsigned row = fp4 ? 32 : 16;   // byte rule of B's rows
        if (!aligned(b, row) || ldb % row != 0) return DG_ERR_ALIGNMENT;
        if (lda < k || ldb < (fp4 ? k / 2 : k)) return DG_ERR_INVALID_ARG;
        const int64_t need = few_workspace_bytes(m, n, k);
        if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return DG_ERR_INVALID_ARG;
        if (need > 0 && !aligned(workspace, 16)) return DG_ERR_ALIGNMENT;
    }
    bool limited = false;
    dg_status st = host_check_device(&sms, &limited);
    if (st != DG_OK) return st;
    cudaError_t e;
    if (k == 0) {
        e = launch_fill_d(c, ldc, d, ldd, m, n, f32, sms, static_cast<cudaStream_t>(stream));
    } else {
        FewParams p = {};
        p.a = static_cast<const uint16_t *>(a);
        p.lda = lda;
        p.b = static_cast<const uint8_t *>(b);
        p.ldb = ldb;
        p.sfb = static_cast<const uint32_t *>(sfb);
        p.c = c;
        p.ldc = ldc;
        p.d = d;
        p.ldd = ldd;
        p.m = m;
        p.n = n;
        p.k = k;
        p.fp4 = fp4;
        p.f32 = f32;
        p.workspace = static_cast<uint8_t *>(workspace);
        p.status = status_dev;
        p.timeout_ns = host_timeout_ns();
        p.debug_flags = host_take_debug_flags();
        e = launch_few_gemv(p, sms, max_occ(limited), static_cast<cudaStream_t>(stream));
    }
    return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

bool layer_unsupported(int t, int topk, int h, int i, int experts) {
    return t > kMaxFewRows || topk > kMaxLayerTopk || experts > kMaxLayerExperts || h > kMaxLayerWidth || i > kMaxLayerWidth;
}

dg_status layer(bool fp4, const void *x, int64_t ldx, const int32_t *ids, const float *weights, const void *w1,
                const void *sf1, const void *w2, const void *sf2, const void *c, int64_t ldc, void *y, int64_t ldy,
                int t, int h, int i, int experts, int topk, void *workspace, int64_t workspace_bytes,
                int32_t *status_dev, void *stream) {
    if (t < 0 || h < 0 || i < 0 || experts < 1 || topk < 1) return DG_ERR_INVALID_ARG;
    if (t == 0 || h == 0) return DG_OK;
    if (layer_unsupported(t, topk, h, i, experts)) return DG_ERR_UNSUPPORTED;
    if (y == nullptr) return DG_ERR_INVALID_ARG;
    if (h % kBlockK != 0 || i % kBlockK != 0) return DG_ERR_ALIGNMENT;
    if (!aligned(y, 16) || ldy % 8 != 0) return DG_ERR_ALIGNMENT;
    if (ldy < h) return DG_ERR_INVALID_ARG;
    if (c != nullptr && (!aligned(c, 16) || ldc % 8 != 0)) return DG_ERR_ALIGNMENT;
    if (c != nullptr && ldc < h) return DG_ERR_INVALID_ARG;
    if (i != 0) {
        if (!x || !ids || !weights || !w1 || !sf1 || !w2 || !sf2 || !workspace) return DG_ERR_INVALID_ARG;
        if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(ids, 4) || !aligned(weights, 4)) return DG_ERR_ALIGNMENT;
        if (ldx < h || workspace_bytes < layer_workspace_bytes(t, topk, h, i, experts)) return DG_ERR_INVALID_ARG;
        const unsigned row = fp4 ? 32 : 16;
        if (!aligned(w1, row) || !aligned(w2, row) || !aligned(sf1, 16) || !aligned(sf2, 16) || !aligned(workspace, 16))
            return DG_ERR_ALIGNMENT;
    }
    int sms = 0;
    bool limited = false;
    dg_status st = host_check_device(&sms, &limited);
    if (st != DG_OK) return st;
    cudaError_t e;
    if (i == 0) {
        e = launch_fill_d(c, ldc, y, ldy, t, h, false, sms, static_cast<cudaStream_t>(stream));
    } else {
        LayerParams p = {};
        p.x = static_cast<const uint16_t *>(x);
        p.ldx = ldx;
        p.ids = ids;
        p.weights = weights;
        p.w1 = static_cast<const uint8_t *>(w1);
        p.sf1 = static_cast<const uint32_t *>(sf1);
        p.w2 = static_cast<const uint8_t *>(w2);
        p.sf2 = static_cast<const uint32_t *>(sf2);
        p.c = static_cast<const uint16_t *>(c);
        p.ldc = ldc;
        p.y = static_cast<uint16_t *>(y);
        p.ldy = ldy;
        p.workspace = static_cast<uint8_t *>(workspace);
        p.t = t;
        p.h = h;
        p.i = i;
        p.experts = experts;
        p.topk = topk;
        p.fp4 = fp4;
        p.status = status_dev;
        p.timeout_ns = host_timeout_ns();
        p.debug_flags = host_take_debug_flags();
        e = launch_moe_layer(p, sms, max_occ(limited), static_cast<cudaStream_t>(stream));
    }
    return e == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_bf16_fp4_gemv_nt(const void *a, int64_t lda, const void *b, int64_t ldb, const void *sfb,
                              const void *c, int64_t ldc, void *d, int64_t ldd, int m, int n, int k,
                              void *workspace, int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    return gemv(true, false, a, lda, b, ldb, sfb, c, ldc, d, ldd, m, n, k, workspace, workspace_bytes, status_dev, stream);
}

dg_status dg_bf16_fp8_gemv_nt(const void *a, int64_t lda, const void *b, int64_t ldb, const void *sfb,
                              const void *c, int64_t ldc, void *d, int64_t ldd, int m, int n, int k,
                              void *workspace, int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    return gemv(false, false, a, lda, b, ldb, sfb, c, ldc, d, ldd, m, n, k, workspace, workspace_bytes, status_dev, stream);
}

dg_status dg_bf16_fp4_gemv_nt_f32(const void *a, int64_t lda, const void *b, int64_t ldb, const void *sfb,
                                  const float *c, int64_t ldc, float *d, int64_t ldd, int m, int n, int k,
                                  void *workspace, int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    return gemv(true, true, a, lda, b, ldb, sfb, c, ldc, d, ldd, m, n, k, workspace, workspace_bytes, status_dev, stream);
}

dg_status dg_bf16_fp8_gemv_nt_f32(const void *a, int64_t lda, const void *b, int64_t ldb, const void *sfb,
                                  const float *c, int64_t ldc, float *d, int64_t ldd, int m, int n, int k,
                                  void *workspace, int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    return gemv(false, true, a, lda, b, ldb, sfb, c, ldc, d, ldd, m, n, k, workspace, workspace_bytes, status_dev, stream);
}

dg_status dg_moe_route(const void *logits, int64_t ld, int logits_fmt, const float *bias, int32_t *ids,
                       float *weights, int t, int experts, int topk, int scoring, int renormalize, float scale,
                       void *stream) {
    if (t < 0 || experts < 1 || topk < 1 || topk > experts) return DG_ERR_INVALID_ARG;
    if (logits_fmt != DG_LOGITS_F32 && logits_fmt != DG_LOGITS_BF16) return DG_ERR_INVALID_ARG;
    if (scoring != DG_SCORE_SOFTMAX && scoring != DG_SCORE_SIGMOID) return DG_ERR_INVALID_ARG;
    if (t > kMaxFewSize || experts > kMaxRouteExperts || topk > kMaxRouteTopk) return DG_ERR_UNSUPPORTED;
    if (t == 0) return DG_OK;
    if (logits == nullptr || ids == nullptr || weights == nullptr || ld < experts) return DG_ERR_INVALID_ARG;
    if (!aligned(logits, logits_fmt == DG_LOGITS_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(bias, 4))
        return DG_ERR_ALIGNMENT;
    int sms = 0;
    bool limited = false;
    dg_status st = host_check_device(&sms, &limited);
    if (st != DG_OK) return st;
    RouteParams p = {logits, ld, bias, ids, weights, t, experts, topk, logits_fmt == DG_LOGITS_BF16,
                     scoring == DG_SCORE_SIGMOID, renormalize != 0, scale, 0};
    return launch_moe_route(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

int64_t dg_bf16_gemv_workspace_bytes(int m, int n, int k) {
    if (m < 0 || n < 0 || k < 0 || m > kMaxFewRows || n > kMaxFewSize || k > kMaxFewSize) return -1;
    return few_workspace_bytes(m, n, k);
}

int64_t dg_moe_layer_workspace_bytes(int t, int topk, int h, int i, int experts) {
    if (t < 0 || topk < 0 || h < 0 || i < 0 || experts < 0 || layer_unsupported(t, topk, h, i, experts)) return -1;
    return layer_workspace_bytes(t, topk, h, i, experts);
}

dg_status dg_moe_fp4_layer(const void *x, int64_t ldx, const int32_t *ids, const float *weights, const void *w1,
                           const void *sf1, const void *w2, const void *sf2, const void *c, int64_t ldc, void *y,
                           int64_t ldy, int t, int h, int i, int experts, int topk, void *workspace,
                           int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    return layer(true, x, ldx, ids, weights, w1, sf1, w2, sf2, c, ldc, y, ldy, t, h, i, experts, topk, workspace,
                 workspace_bytes, status_dev, stream);
}

dg_status dg_moe_fp8_layer(const void *x, int64_t ldx, const int32_t *ids, const float *weights, const void *w1,
                           const void *sf1, const void *w2, const void *sf2, const void *c, int64_t ldc, void *y,
                           int64_t ldy, int t, int h, int i, int experts, int topk, void *workspace,
                           int64_t workspace_bytes, int32_t *status_dev, void *stream) {
    return layer(false, x, ldx, ids, weights, w1, sf1, w2, sf2, c, ldc, y, ldy, t, h, i, experts, topk, workspace,
                 workspace_bytes, status_dev, stream);
}

}  // extern "C"
