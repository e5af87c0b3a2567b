// Launches of the few-row kernel (few_rows.cuh): tile and split choice, tensor maps.
//
// The times beside the rules are of these kernels, both sides of a rule in one run: microseconds a call
// over calls in a row in a CUDA graph, on weights that are not in L2, the median of three graphs' medians.
// They repeat within 1.5 % on one GPU, and between GPUs within 3 %.
#include "few_rows.cuh"

#include <atomic>
#include <mutex>

namespace dg {
namespace {

constexpr int kMaxSplit = 8;        // portable cluster size
// Tokens of a layer's segment: 64 in three pieces, their scales and 64 tokens' results would take 272
// columns of TMEM, and two CTAs have 256 each.
constexpr int kMaxSegment = 32;
// Shared memory of a CTA, alone on an SM or one of two.  It also keeps CTAs apart that would want
// more TMEM than there is: of a kernel and the one that starts beside its end, the later CTA
// could take the columns that the earlier one has yet to allocate, and then wait for it.  Two CTAs
// take up to 256 columns each and leave no room for a third, nor for one of the GEMM kernels,
// which take all 512 and over 116 KB.
constexpr int kSmemOne = 232448 - 1024, kSmemTwo = 114000;
static_assert(kSmemTwo + 116 * 1024 + 2 * 1024 > 228 * 1024, "no room beside a kernel that takes all of TMEM");

// Bytes of weights an SM brings to L2 before it waits for the preceding kernel (FP4, 1 x 2112 x 7168
// 4.75 us without, 4.42 us with; 1 x 24576 x 1536 6.32 and 6.01).
constexpr int kAhead = 160 * 1024;

int cdiv(int a, int b) { return (a + b - 1) / b; }
int pow2_at_least(int v) {
    int p = 32;
    while (p < v) p *= 2;
    return p;
}

// Rows of weights seen as [rows / 4][4]: weight row 4l + c lands in operand row 32c + l.
bool encode_weights(CUtensorMap *map, int w, const void *base, int64_t rows, int64_t ld_bytes, int k) {
    const TensorMapEncodeFn enc = host_encode();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(w == kFp4Packed ? k / 2 : k), static_cast<cuuint64_t>(rows / 4), 4};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(4 * ld_bytes), static_cast<cuuint64_t>(ld_bytes)};
    const cuuint32_t box[3] = {128, 32, 4};
    const cuuint32_t step[3] = {1, 1, 1};
    return enc(map, w == kFp4 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
               const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a launch fills the GPU: `occ` CTAs on an SM; `split` CTAs of a cluster share a
// tile's K (1: persistent CTAs take the tiles in turn).
struct Plan {
    int occ, split;
};

template <int W, int HALVES, int MODE>
cudaError_t launch(const CUtensorMap &map, FewArgs &a, const Plan &plan, int max_tiles,
                   int num_sms, cudaStream_t stream) {
    const int tables = MODE < kUp ? 0 : segment_table_bytes(a.tokens * a.topk, a.experts);
    a.out_bytes = FewConfig::out_bytes(HALVES, MODE, a.tokens, plan.split);
    a.ahead = kAhead / (HALVES * (W == kFp4 ? 8192 : 16384)) / plan.occ;
    const int tokens = a.tokens < a.cap ? a.tokens : a.cap;   // of a tile, at most
    constexpr int pieces = MODE == kDown ? inner_pieces(W) : pieces_of(W);
    a.b_rows = FewConfig::b_rows(pieces, tokens);
    const int stage = FewConfig::stage_bytes(W, HALVES, a.b_rows), limit = plan.occ == 2 ? kSmemTwo : kSmemOne;
    const int ring = limit - FewConfig::fixed_bytes(tables);
    // Split results of more than 8 KB go to the ring where they would cost a stage: one more wait
    // instead (17 x 4096 x 7168 FP8, at no stage, 10.8 us so and 10.4 us beside the ring; MoE layer of 64 tokens,
    // top 8 of 64 experts, 7168 x 2048 FP4, down kernel with a ring of 3 256 us so and 298 us beside one of 2).
    if (plan.split > 1 && a.out_bytes > 8192 && (ring - a.out_bytes) / stage < ring / stage) a.out_bytes = 0;
    int stages = (ring - a.out_bytes) / stage;
    if (stages > FewConfig::kMaxStages) stages = FewConfig::kMaxStages;
    if (stages < 2) return cudaErrorInvalidConfiguration;
    const int set = HALVES * FewConfig::b_rows(pieces, a.cap), most = plan.occ == 2 ? 256 : 512;
    const int sf = 2 * HALVES * 8 * scale_blocks(W) + (MODE == kDown ? HALVES * ((a.tokens + 7) & ~7) : 0);
    a.stages = stages;
    a.accs = (plan.split == 1 || MODE == kDown) && 2 * set + sf <= most ? 2 : 1;
    a.tmem_cols = pow2_at_least(a.accs * set + sf);
    if (a.tmem_cols > (plan.occ == 2 ? 256 : 512)) return cudaErrorInvalidConfiguration;
    const int smem = limit;   // (all of it, whatever the stages take: see kSmemTwo)
    auto kernel = dg_few_rows_kernel<W, HALVES, MODE>;
    static std::atomic<uint64_t> ready{0};   // devices whose attributes are set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(ready.load() >> (dev & 63) & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess) ready.fetch_or(uint64_t{1} << (dev & 63));
    }
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
    cfg.blockDim = dim3(FewConfig::threads(W, HALVES, MODE, a.tokens));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = plan.split > 1 ? 2 : 1;
    host_set_last_config(HALVES * 128, a.b_rows, stages, grid, MODE < kUp ? 3 : 5,
                         MODE == kGemv ? 1 : MODE < kDown ? 2 : a.launches);
    return cudaLaunchKernelEx(&cfg, kernel, map, a);
}

template <int HALVES, int MODE>
cudaError_t launch_fmt(int w, const CUtensorMap &map, FewArgs &a, const Plan &plan, int max_tiles, int num_sms,
                       cudaStream_t stream) {
    if (w == kFp8) return launch<kFp8, HALVES, MODE>(map, a, plan, max_tiles, num_sms, stream);
    if (w == kFp4Packed) return launch<kFp4Packed, HALVES, MODE>(map, a, plan, max_tiles, num_sms, stream);
    // (rows few enough for a kernel to split them itself have their FP4 weights packed)
    if constexpr (!splits_itself(MODE)) return launch<kFp4, HALVES, MODE>(map, a, plan, max_tiles, num_sms, stream);
    return cudaErrorInvalidValue;
}

// Clusters of 1..kMaxSplit CTAs that are resident at once with one CTA on an SM (the SMs
// of a cluster lie in one GPC, so the larger ones leave SMs over).
const int *resident_clusters(int num_sms) {
    static int count[64][kMaxSplit + 1];
    static bool ready[64];
    static std::mutex mutex;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    dev &= 63;
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
        auto kernel = dg_few_rows_kernel<kFp8, 1, kGemv>;
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
        for (int c = 1; c <= kMaxSplit; ++c) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(c);
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(static_cast<unsigned>(c * num_sms));
            cfg.blockDim = dim3(FewConfig::threads(kFp8, 1, kGemv));
            cfg.dynamicSmemBytes = kSmemOne;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
            count[dev][c] = n;
        }
        cudaGetLastError();   // a failed query means no clusters, not an error
        ready[dev] = true;
    }
    return count[dev];
}

// Cluster size for `tiles` tiles of `kblocks` K-blocks: of those whose clusters are all
// resident at once, the one with the least K-blocks on the busiest SM, the larger of equals
// (more of the latency of a CTA's start and end overlaps).  Where an SM would have one CTA in the
// room of two, its K-blocks count 1.6 times, for it has half a ring: 17 x 6144 x 8192 FP4 12.1 us in
// clusters of 3 (144 CTAs) and 10.6 us of 5 (240), 1 x 4096 x 7168 5.6 us of 4 and 5.2 of 6 (64 x 4096 x
// 2048 9.1 and 9.5); the layer's down kernel, 64 tokens, h = 6400: 275 us of 3 and 244 of 5.  A second wave
// of clusters costs more than any split gains (24576 x 1536, 192 tiles: 5.9 us unsplit, 8.7 us in pairs).
// `tight`: whether clusters may take all of that residence.  A kernel starts while CTAs of
// the ones around it still hold SMs, and clusters that find no room then make a second wave,
// which costs most where a CTA has little to do (1 x 7168 x 2048, 56 tiles in clusters of 5, 2 K-blocks
// a CTA: 5.2 us, 4.3 us in clusters of 4; the layer's down kernel, h = 7168: 326 and 256 us).  With more to
// do, clusters of up to 4 find their room: 72 tiles of 16 x 9216 x 4096 FP4 take 8.9 us in clusters of 4 and
// 9.3 us of 3; larger ones need that many free SMs of one GPC at once and often do not: 1 x 7168 x 16384
// 14.4 us in clusters of 5 and 12.4 us of 4 (FP8 24.9 and 20.9; 16 rows 16.5 and 17.1).
int choose_split(int tiles, int64_t kblocks, int occ, int num_sms, bool tight) {
    const int *clusters = resident_clusters(num_sms);
    int best = 1;
    int64_t best_cost = -1;
    for (int s = 1; s <= kMaxSplit && s <= kblocks; ++s) {
        const bool full = tight && kblocks >= 8 * s;
        const bool fits = full ? tiles < clusters[s] * occ + (s <= 4) : tiles * 10 <= clusters[s] * occ * 9;
        if (s > 1 && (!fits || tiles * s > occ * num_sms)) continue;
        const int on_sm = cdiv(tiles * s, num_sms);
        const int64_t cost = (on_sm < occ ? 8 : 5 * on_sm) * ((kblocks + s - 1) / s);
        if (best_cost < 0 || cost <= best_cost) { best = s; best_cost = cost; }
    }
    return best;
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

// Rows that every CTA of a product splits by itself, without the split kernel's launch and
// workspace.  FP8, 3 rows, 2112 x 7168: 5.6 us so and 7.4 us with it, 8 rows 6.3 and 7.6 us (4096
// x 7168 8.3 and 9.6, 65536 x 7168 74.8 and 75.3, 12 rows 94 and 77 us).  The eight digits of
// FP4's take longer: 2 rows, 4096 x 7168 5.7 us so and 7.4 with it, 65536 x 7168 40.2 and 41.3; 3 rows
// 7.3 and 7.6, 46.1 and 41.2; 8 rows, 4096 x 7168 10.6 and 7.9 us.
bool direct(int w, int64_t m) { return m <= (w == kFp4Packed ? 2 : 8); }

int capacity(int tokens) { return tokens <= 8 ? 8 : tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64; }

// Tokens of a segment at most: room for twice the mean number of tokens of an expert (the
// tokens beyond make another segment, which reads the expert's weights again).  Less room
// leaves more of the ring to the weights, and up to 8 tokens their packed form.  Top 8 of 64 experts,
// routed evenly, 64 tokens (mean 8), 7168 x 2048 FP4: 256 us with room for 16, 305 us for 32 and 273 us
// for 8; 4096 x 1024 FP8 140, 147 and 149 us; 32 tokens, 7168 x 2048 FP4: 235 us with room for 8, 243 for 16.
int segment_capacity(int64_t t, int64_t topk, int64_t experts) {
    const int64_t most = 2 * t * topk / experts;
    const int cap = capacity(static_cast<int>(most < t ? most : t));
    return cap < kMaxSegment ? cap : kMaxSegment;
}

// Parts of an expert's K-blocks in the down kernel, each for one CTA of a cluster.  Short parts are narrow
// strips of many weight rows, and take longer a K-block (413 ns with parts of 6 on 128 CTAs, 458 ns of
// 3, 625 ns of one), so parts are of 3 at least; with fewer parts the CTAs' shares are less even.  7 tokens, top 6 of 64 experts,
// 2048 x 1408 FP4 (6 K-blocks, clusters of 8): 38.6 us in one part, 37.1 in 2, 38.3 in 3, 40.0 in 6;
// FP8 (11): 59.3 in one, 55.7 in 3, 57.4 in 6; 64 tokens, top 8 of 256, 4096 x 1024 FP4 (4 of 6): 254 in
// one, 248 in 2, 262 in 4; 24 tokens, top 5 of 48, 3584 x 640 (3 of 5): 47 in one, 52 in 3.
int down_parts(int kblocks, int split) {
    const int parts = kblocks / 3;
    return parts < 1 ? 1 : parts < split ? parts : split;
}

// FP4 weights packed, where all activations fit the digits' 64 columns: 8 x 131064 x 7168 79.2 us,
// 83.5 us unpacked; one row 77.1 and 82.8; MoE layer of one token, top 8 of 64 experts, 7168 x 2048, 37.2 us
// packed and 38.3 us unpacked, of 64 tokens and 256 experts, 4096 x 1024, 254 and 263 us.
int format_of(bool fp4, int cap) { return !fp4 ? kFp8 : cap == 8 ? kFp4Packed : kFp4; }

// Bounds of the layer's segments and of their images.
struct SegmentBounds {
    int w, cap;
    int64_t count, units, inner_units;
    SegmentBounds(bool fp4, int64_t t, int64_t topk, int64_t experts) {
        const int64_t pairs = t * topk, used = pairs < experts ? pairs : experts;
        cap = segment_capacity(t, topk, experts);
        w = format_of(fp4, cap);
        count = used + pairs / cap;
        if (count > pairs) count = pairs;
        // (up to 8 tokens: a segment takes the room of all tokens)
        units = w == kFp4Packed ? pairs : t <= 8 ? count * image_units(pieces_of(w), static_cast<int>(t))
                                                 : (pairs + 3 * count) / 4;
        inner_units = inner_units_before(w, static_cast<int>(pairs), static_cast<int>(count));
    }
    int64_t blocks(int64_t k) const { return (k + block_k(w) - 1) / block_k(w); }
    int64_t image(int64_t k) const { return units * blocks(k) * 1024; }
    int64_t inner_image(int64_t k) const { return inner_units * blocks(k) * 1024; }
    int64_t scales(int64_t k) const { return count * blocks(k) * scale_blocks(w) * 512; }
};

}  // namespace

int64_t few_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    int64_t most = 0;   // of either weight type
    for (int w : {static_cast<int>(kFp8), format_of(true, capacity(static_cast<int>(m)))}) {
        if (direct(w, m)) continue;
        const int64_t blocks = (k + block_k(w) - 1) / block_k(w);
        const int64_t bytes = blocks * (image_units(pieces_of(w), static_cast<int>(m)) * 1024 + scale_blocks(w) * 512);
        if (bytes > most) most = bytes;
    }
    return most;
}

int64_t layer_workspace_bytes(int64_t t, int64_t topk, int64_t h, int64_t i, int64_t experts) {
    if (t == 0 || topk == 0 || experts == 0 || h == 0 || i == 0) return 0;   // nothing to split
    int64_t most = 0;
    for (bool fp4 : {false, true}) {
        const SegmentBounds b(fp4, t, topk, experts);
        const int64_t bytes = b.image(h) + b.inner_image(i) + b.scales(h) + b.scales(i);
        if (bytes > most) most = bytes;
    }
    return most;
}

cudaError_t launch_few_gemv(const FewParams &p, int num_sms, int max_occ, cudaStream_t stream) {
    FewArgs a = {};
    a.cap = capacity(p.m);
    const int w = format_of(p.fp4, a.cap);
    CUtensorMap map;
    if (!encode_weights(&map, w, p.b, p.n, p.ldb, p.k)) return cudaErrorInvalidValue;
    a.x = p.a;
    a.ldx = p.lda;
    a.sf = p.sfb;
    a.sf_ld = cdiv(p.n, 4) * 4;
    a.rows = p.n;
    a.tokens = p.m;
    a.kblocks = cdiv(p.k, block_k(w));
    a.slices = p.fp4 ? p.k / 128 : cdiv(p.k, 512);
    a.last_mmas = p.k % 256 ? 2 : 4;
    a.c = p.c;
    a.ldc = p.ldc;
    a.d = p.d;
    a.ldd = p.ldd;
    a.f32 = p.f32;
    a.status = p.status;
    a.timeout_ns = p.timeout_ns;
    a.debug_flags = p.debug_flags;
    // The split of K depends on n, k, the format and dg_set_num_sms alone, so a row's result does not
    // depend on the other rows of the call.
    a.row_tiles = cdiv(p.n, 128);
    Plan plan = {max_occ, choose_split(a.row_tiles, a.kblocks, max_occ, num_sms, true)};
    // Many tiles: two CTAs on an SM, except where, after whole rounds of them, so few tiles are left
    // that an SM has one, and its ring is half as deep as one CTA's.  1024 tiles (131064 x 7168
    // FP4, 112 left): two CTAs 82.3 and one 79.0 us at 8 rows, 91.1 and 85.3 at 16; 512 (208 left): 48.2
    // and 50.8 at 16 rows; 352 (48 left) 43.5 and 39.2.  Rings of two CTAs are too short beside more
    // than 32 rows: 64 rows, 1024 tiles 120 and 105 us, 512 tiles 64.2 and 61.8.  With one round
    // (192 tiles) two CTAs are better all the same: 32.3 and 33.8 us at 64 rows; and where CTAs split
    // the rows themselves: 61.6 and 67.8 us at 8 rows of FP8, 352 tiles.
    const int left = a.row_tiles % (2 * num_sms);
    if (plan.split == 1 && a.row_tiles > 2 * num_sms && !direct(w, p.m) && (p.m > 32 || (left > 0 && left <= num_sms)))
        plan.occ = 1;
    if (direct(w, p.m)) return launch_fmt<1, kGemv>(w, map, a, plan, a.row_tiles, num_sms, stream);
    uint8_t *image = p.workspace;
    uint8_t *image_sf = image + static_cast<int64_t>(a.kblocks) * image_units(pieces_of(w), p.m) * 1024;
    const int rows = 256 * 8 / block_k(w);   // rows' K-blocks of a CTA
    Dependent split(dim3(static_cast<unsigned>(cdiv(p.m * a.kblocks, rows))), 0, stream);
    cudaError_t e = cudaLaunchKernelEx(&split.cfg, w == kFp4Packed ? dg_few_split_kernel<kFp4Packed> : dg_few_split_kernel<kFp8>,
                                       a.x, a.ldx, p.m, p.k, image, image_sf);
    if (e != cudaSuccess) return e;
    a.image = image;
    a.image_sf = image_sf;
    return launch_fmt<1, kGemvPre>(w, map, a, plan, a.row_tiles, num_sms, stream);
}

cudaError_t launch_moe_layer(const LayerParams &p, int num_sms, int max_occ, cudaStream_t stream) {
    const SegmentBounds bounds(p.fp4, p.t, p.topk, p.experts);
    const int w = bounds.w, cap = bounds.cap, pairs = p.t * p.topk;
    CUtensorMap map1, map2;
    const int64_t per = p.fp4 ? 2 : 1;
    if (!encode_weights(&map1, w, p.w1, static_cast<int64_t>(p.experts) * 2 * p.i, p.h / per, p.h) ||
        !encode_weights(&map2, w, p.w2, static_cast<int64_t>(p.experts) * p.h, p.i / per, p.i))
        return cudaErrorInvalidValue;
    uint8_t *x_image = p.workspace, *h_image = x_image + bounds.image(p.h);
    uint8_t *x_sf = h_image + bounds.inner_image(p.i), *h_sf = x_sf + bounds.scales(p.h);
    const int kh = static_cast<int>(bounds.blocks(p.h)), ki = static_cast<int>(bounds.blocks(p.i));
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
    const int down_tiles = cdiv(p.h, 128);
    // The split of K depends on h, i, the number of experts, the weights' form and dg_set_num_sms
    // alone, and the up kernel does not split it, so a token's result does not depend on the other tokens.
    const Plan down = {max_occ, choose_split(down_tiles, static_cast<int64_t>(ki) * p.experts, max_occ, num_sms, false)};
    // up: a tile is 128 columns of h of one segment
    a.image = x_image;
    a.image_sf = x_sf;
    a.out_image = h_image;
    a.out_image_sf = h_sf;
    a.sf = p.sf1;
    a.sf_ld = 2 * p.i;
    a.slices = p.fp4 ? p.h / 128 : cdiv(p.h, 512);
    a.last_mmas = p.h % 256 ? 2 : 4;
    a.sf_expert = static_cast<int64_t>(a.slices) * a.sf_ld;
    a.rows = 2 * p.i;
    a.kblocks = kh;
    a.row_tiles = p.i / 128;
    // K is not split: a token alone would then have its sums split otherwise than among many.  (Measured
    // before that form was taken out, it gains only where tiles are few and K is long: 1 token, top 1, 5120 x 2048 FP8 20.5 us so and 15.6 us in
    // clusters of 6, top 2, 7168 x 2048 FP4 19.3 and 17.2; top 8 of 128, 2048 x 768 13.9 and 15.3, top 6
    // of 64, 2048 x 1408 15.1 and 16.5.)
    const int up_tiles = static_cast<int>(bounds.count) * a.row_tiles;
    const Plan up = {1, 1};
    // With no more tokens than experts, counting a token once per slot, the up kernel splits x
    // itself, a launch less: 1 token, top 8 of 64 experts, 7168 x 2048 FP4 37.3 us so and 39.7 us
    // with the split kernel, FP8 (of 32) 59.1 and 60.3 us, 2 tokens, top 2 of 8, 1024 x 512 9.3
    // and 10.0 us, 7 tokens, top 6 of 64, 2048 x 1408 37.3 and 39.1.  With more its own splitting bounds
    // it: 8 tokens, top 4 of 8 experts, 7168 x 2048 FP4 47 us so and 43 us with the split kernel, 16
    // tokens, top 4 of 16 89 and 73 us (FP8, whose pieces take less, 16 tokens, top 8 of 32: 211 and 215).
    cudaError_t e;
    if (pairs <= p.experts) {
        a.x = p.x;
        a.ldx = p.ldx;
        a.launches = 2;
        e = launch_fmt<2, kUpSelf>(w, map1, a, up, up_tiles, num_sms, stream);
    } else {
        const int rows = 256 * 8 / block_k(w);
        Dependent split(dim3(static_cast<unsigned>(kh), static_cast<unsigned>(cdiv(pairs, 4 * rows))),
                        segment_table_bytes(pairs, p.experts), stream);
        e = cudaLaunchKernelEx(&split.cfg,
                               w == kFp4Packed ? dg_layer_split_kernel<kFp4Packed> : dg_layer_split_kernel<kFp8>,
                               p.x, p.ldx, p.ids, p.t, p.topk, p.experts, cap, p.h, x_image, x_sf);
        if (e != cudaSuccess) return e;
        a.launches = 3;
        e = launch_fmt<2, kUp>(w, map1, a, up, up_tiles, num_sms, stream);
    }
    if (e != cudaSuccess) return e;
    // down: K runs over the segments
    a.row_tiles = down_tiles;
    a.image = h_image;
    a.image_sf = h_sf;
    a.sf = p.sf2;
    a.sf_ld = p.h;
    a.slices = p.fp4 ? p.i / 128 : cdiv(p.i, 512);
    a.last_mmas = p.i % 256 ? 2 : 4;
    a.sf_expert = static_cast<int64_t>(a.slices) * a.sf_ld;
    a.rows = p.h;
    a.kblocks = ki;
    a.parts = down_parts(ki, down.split);
    a.c = p.c;
    a.ldc = p.ldc;
    a.d = p.y;
    a.ldd = p.ldy;
    a.debug_flags = 0;
    return launch_fmt<1, kDown>(w, map2, a, down, a.row_tiles, num_sms, stream);
}

}  // namespace dg
