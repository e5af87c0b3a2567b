// Launches of the few-row kernel (few_rows.cuh): tile and split choice, tensor maps.
#include "few_rows.cuh"

#include <cstdlib>

namespace dg {
namespace {

constexpr int kMaxSplit = 8;        // portable cluster size
constexpr int kSmemOne = 232448 - 1024, kSmemTwo = 114000;   // bytes for one or two CTAs on an SM

int cdiv(int a, int b) { return (a + b - 1) / b; }
int pow2_at_least(int v) {
    int p = 32;
    while (p < v) p *= 2;
    return p;
}
int env(const char *n, int d) { const char *e = std::getenv(n); return e ? std::atoi(e) : d; }

// Rows of weights seen as [rows / 4][4]: weight row 4l + c lands in operand row 32c + l.
bool encode_weights(CUtensorMap *map, bool fp4, const void *base, int64_t rows, int64_t ld_bytes, int k) {
    const TensorMapEncodeFn enc = host_encode();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows / 4), 4};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(4 * ld_bytes), static_cast<cuuint64_t>(ld_bytes)};
    const cuuint32_t box[3] = {128, 32, 4};
    const cuuint32_t step[3] = {1, 1, 1};
    return enc(map, fp4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
               const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a launch fills the GPU: `occ` CTAs on an SM; `split` CTAs of a cluster share a
// tile's K (1: persistent CTAs take the tiles in turn).
struct Plan {
    int halves, occ, split;
};

template <bool FP4, int HALVES, int MODE>
cudaError_t launch(const CUtensorMap &map, FewArgs &a, const Plan &plan, int max_tiles,
                   int num_sms, cudaStream_t stream) {
    const int tables = MODE < kUp ? 0 : segment_table_bytes(a.tokens * a.topk, a.experts);
    const int fixed = FewConfig::smem_bytes(HALVES, a.cap, 0, MODE, plan.split, tables);
    const int stage = FewConfig::stage_bytes(HALVES, a.cap);
    const int limit = plan.occ == 2 ? kSmemTwo : kSmemOne;
    int stages = (limit - fixed) / stage;
    if (stages > FewConfig::kMaxStages) stages = FewConfig::kMaxStages;
    if (stages > env("DG_ST", 99)) stages = env("DG_ST", 99);
    if (stages < 2) return cudaErrorInvalidConfiguration;
    const int set = HALVES * 2 * a.cap, most = plan.occ == 2 ? 256 : 512;
    const int sf = 2 * HALVES * 8 + (MODE == kDown ? HALVES * ((a.tokens + 7) & ~7) : 0);
    a.stages = stages;
    a.accs = (plan.split == 1 || MODE == kDown) && 2 * set + sf <= most ? 2 : 1;
    a.tmem_cols = pow2_at_least(a.accs * set + sf);
    if (a.tmem_cols > 512) return cudaErrorInvalidConfiguration;
    const int smem = FewConfig::smem_bytes(HALVES, a.cap, stages, MODE, plan.split, tables);
    auto kernel = dg_few_rows_kernel<FP4, HALVES, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    const int grid = plan.split > 1 ? max_tiles * plan.split
                                    : (max_tiles < plan.occ * num_sms ? max_tiles : plan.occ * num_sms);
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(FewConfig::threads(HALVES, MODE));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = plan.split > 1 ? 2 : 1;
    host_set_last_config(HALVES * 128, 2 * a.cap, stages, grid, MODE < kUp ? 3 : 5,
                         MODE == kGemv ? 1 : MODE == kGemvPre ? 2 : 3);
    return cudaLaunchKernelEx(&cfg, kernel, map, a);
}

template <int HALVES, int MODE>
cudaError_t launch_fmt(bool fp4, const CUtensorMap &map, FewArgs &a, const Plan &plan, int max_tiles, int num_sms,
                       cudaStream_t stream) {
    return fp4 ? launch<true, HALVES, MODE>(map, a, plan, max_tiles, num_sms, stream)
               : launch<false, HALVES, MODE>(map, a, plan, max_tiles, num_sms, stream);
}

template <int MODE>
cudaError_t launch_mode(bool fp4, const CUtensorMap &map, FewArgs &a, const Plan &plan, int max_tiles, int num_sms,
                        cudaStream_t stream) {
    return plan.halves == 2 ? launch_fmt<2, MODE>(fp4, map, a, plan, max_tiles, num_sms, stream)
                            : launch_fmt<1, MODE>(fp4, map, a, plan, max_tiles, num_sms, stream);
}

// The largest cluster of at most kMaxSplit CTAs (and K-blocks) with all tiles resident at once.
int resident_split(int tiles, int kblocks, int slots) {
    int s = slots / tiles;
    if (s > kMaxSplit) s = kMaxSplit;
    if (s > kblocks) s = kblocks;
    return s < 1 ? 1 : s;
}

// A launch that may start before the stream's previous kernel ends.
struct Dependent {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    Dependent(dim3 grid, int smem, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = grid;
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

// Rows that a product splits by itself (each CTA its own K range).
bool direct(int64_t m) { return m <= env("DG_FEW_DIRECT", 4); }

int capacity(int tokens) { return tokens <= 8 ? 8 : tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64; }

// Tokens of a segment at most: room for twice the mean number of tokens of an expert (the
// tokens beyond make another segment, which reads the expert's weights again).
int segment_capacity(int64_t t, int64_t topk, int64_t experts) {
    const int64_t most = 2 * t * topk / experts + 4;
    return capacity(static_cast<int>(most < t ? most : t));
}

// Bounds of the layer's segments, and of their units of 8 image rows (4 tokens).
struct SegmentBounds {
    int64_t count, units;
    SegmentBounds(int64_t t, int64_t topk, int64_t experts) {
        const int64_t pairs = t * topk, used = pairs < experts ? pairs : experts;
        const int cap = segment_capacity(t, topk, experts);
        count = used + pairs / cap;
        if (count > pairs) count = pairs;
        units = (pairs + 3 * count) / 4;
    }
    int64_t image(int64_t k) const { return units * (k / 128) * 1024; }
    int64_t scales(int64_t k) const { return count * (k / 128) * 512; }
};

}  // namespace

int64_t few_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    return direct(m) ? 0 : k / 128 * ((m + 3) / 4 * 1024 + 512);
}

int64_t layer_workspace_bytes(int64_t t, int64_t topk, int64_t h, int64_t i, int64_t experts) {
    if (t == 0 || topk == 0 || experts == 0) return 0;
    const SegmentBounds b(t, topk, experts);
    return b.image(h) + b.image(i) + b.scales(h) + b.scales(i);
}

cudaError_t launch_few_gemv(const FewParams &p, int num_sms, cudaStream_t stream) {
    CUtensorMap map;
    if (!encode_weights(&map, p.fp4, p.b, p.n, p.ldb, p.k)) return cudaErrorInvalidValue;
    FewArgs a = {};
    a.x = p.a;
    a.ldx = p.lda;
    a.sf = p.sfb;
    a.sf_ld = cdiv(p.n, 4) * 4;
    a.rows = p.n;
    a.tokens = p.m;
    a.kblocks = p.k / 128;
    a.cap = capacity(p.m);
    a.c = p.c;
    a.ldc = p.ldc;
    a.d = p.d;
    a.ldd = p.ldd;
    a.f32 = p.f32;
    a.status = p.status;
    a.timeout_ns = p.timeout_ns;
    a.debug_flags = p.debug_flags;
    Plan plan;
    plan.halves = env("DG_H", p.m > 16 ? 2 : 1);
    plan.occ = env("DG_OCC", plan.halves == 1 ? 2 : 1);
    plan.split = env("DG_S", resident_split(cdiv(p.n, 128), a.kblocks, 2 * num_sms * 19 / 20));
    a.row_tiles = cdiv(p.n, 128 * plan.halves);
    if (direct(p.m)) return launch_mode<kGemv>(p.fp4, map, a, plan, a.row_tiles, num_sms, stream);
    a.image = p.workspace;
    a.image_sf = p.workspace + static_cast<int64_t>(a.kblocks) * ((p.m + 3) / 4) * 1024;
    Dependent split(dim3(static_cast<unsigned>(cdiv(p.m * a.kblocks, 16))), 0, stream);
    cudaError_t e = cudaLaunchKernelEx(&split.cfg, dg_few_split_kernel, a.x, a.ldx, p.m, a.kblocks,
                                       const_cast<uint8_t *>(a.image), const_cast<uint8_t *>(a.image_sf));
    if (e != cudaSuccess) return e;
    return launch_mode<kGemvPre>(p.fp4, map, a, plan, a.row_tiles, num_sms, stream);
}

cudaError_t launch_moe_layer(const LayerParams &p, int num_sms, cudaStream_t stream) {
    CUtensorMap map1, map2;
    const int64_t per = p.fp4 ? 2 : 1;
    if (!encode_weights(&map1, p.fp4, p.w1, static_cast<int64_t>(p.experts) * 2 * p.i, p.h / per, p.h) ||
        !encode_weights(&map2, p.fp4, p.w2, static_cast<int64_t>(p.experts) * p.h, p.i / per, p.i))
        return cudaErrorInvalidValue;
    const SegmentBounds bounds(p.t, p.topk, p.experts);
    uint8_t *x_image = p.workspace, *h_image = x_image + bounds.image(p.h);
    uint8_t *x_sf = h_image + bounds.image(p.i), *h_sf = x_sf + bounds.scales(p.h);
    const int cap = segment_capacity(p.t, p.topk, p.experts), pairs = p.t * p.topk;
    const int kh = p.h / 128, ki = p.i / 128;
    Dependent split(dim3(static_cast<unsigned>(kh), static_cast<unsigned>(cdiv(pairs, 64))),
                    segment_table_bytes(pairs, p.experts), stream);
    cudaError_t e = cudaLaunchKernelEx(&split.cfg, dg_layer_split_kernel, p.x, p.ldx, p.ids, p.t, p.topk, p.experts,
                                       cap, kh, x_image, x_sf);
    if (e != cudaSuccess) return e;
    FewArgs a = {};
    a.tokens = p.t;
    a.cap = cap;
    a.ids = p.ids;
    a.weights = p.weights;
    a.experts = p.experts;
    a.topk = p.topk;
    a.inner = p.i;
    a.status = p.status;
    a.timeout_ns = p.timeout_ns;
    a.debug_flags = p.debug_flags;
    // up: a tile is 128 columns of h of one segment
    a.image = x_image;
    a.image_sf = x_sf;
    a.out_image = h_image;
    a.out_image_sf = h_sf;
    a.sf = p.sf1;
    a.sf_ld = 2 * p.i;
    a.sf_expert = static_cast<int64_t>(p.fp4 ? kh : cdiv(kh, 4)) * a.sf_ld;
    a.rows = 2 * p.i;
    a.kblocks = kh;
    a.row_tiles = ki;
    const int up_tiles = static_cast<int>(bounds.count) * ki;
    Plan up;
    up.halves = 2;
    up.occ = env("DG_UP_OCC", 1);
    up.split = env("DG_UP_S", resident_split(up_tiles, kh, up.occ * num_sms * 19 / 20));
    e = launch_fmt<2, kUp>(p.fp4, map1, a, up, up_tiles, num_sms, stream);
    if (e != cudaSuccess) return e;
    // down: K runs over the segments
    a.image = h_image;
    a.image_sf = h_sf;
    a.sf = p.sf2;
    a.sf_ld = p.h;
    a.sf_expert = static_cast<int64_t>(p.fp4 ? ki : cdiv(ki, 4)) * a.sf_ld;
    a.rows = p.h;
    a.kblocks = ki;
    a.c = p.c;
    a.ldc = p.ldc;
    a.d = p.y;
    a.ldd = p.ldy;
    a.debug_flags = 0;
    Plan down;
    down.halves = env("DG_DOWN_H", 1);
    down.occ = env("DG_DOWN_OCC", p.t > 16 ? 1 : 2);
    a.row_tiles = cdiv(p.h, 128 * down.halves);
    down.split = env("DG_DOWN_S", resident_split(a.row_tiles, ki * static_cast<int>(bounds.count),
                                                 down.occ * num_sms * 19 / 20));
    return launch_mode<kDown>(p.fp4, map2, a, down, a.row_tiles, num_sms, stream);
}

}  // namespace dg
