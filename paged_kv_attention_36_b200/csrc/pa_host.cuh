// pa_host.cuh -- host-side pieces shared by the translation units of the
// library: checks, device queries, workspace layout and tensor maps.  All of
// it has internal linkage.
#pragma once

#include <cudaTypedefs.h>

#include <cstdlib>
#include <cstring>
#include <mutex>

#include "pa_decode.cuh"
#include "pa_prefill_tc.cuh"

namespace pa {
// read_error_word() of pa_serving.cu's kernels (defined there).
bool serving_error_word(unsigned int* bits, bool clear);
}  // namespace pa

namespace {

constexpr int kBlockSize = 16;  // tokens per physical block the decode kernels are built for
constexpr int kMinPagesPerCta = 2;  // pages of a head group: fewest worth a CTA
constexpr int kMaxDevices = 64;
constexpr int kMaxCtas = 1024;  // the two-level split merge handles up to 16 x 64 pieces
constexpr float kLog2e = 1.4426950408889634f;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// This translation unit's device error word, read and cleared (synchronous).
bool read_error_word(unsigned int* bits, bool clear) {
    if (cudaMemcpyFromSymbol(bits, pa::g_device_errors, sizeof *bits) != cudaSuccess) return false;
    const unsigned int zero = 0;
    return !clear || cudaMemcpyToSymbol(pa::g_device_errors, &zero, sizeof zero) == cudaSuccess;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The math policies: tensor-core (default) or fp32 CUDA-core for bf16
// caches; tensor-core for fp8 (E4M3) caches.
enum class MathKind { kMma, kSimt, kFp8 };

#ifndef PA_MAX_RING
#define PA_MAX_RING 64
#endif
// Deepest ring of stages whose CTA fits in shared memory, a multiple of
// the most stages a page can take (with 32 KB stages: 7 at head_dim 64,
// 6 at 128).
template <int D, int EB = 2>
constexpr int ring_fit() {
    using C1 = pa::DecodeCfg<D, kBlockSize, 1, EB>;
    int r = PA_MAX_RING;
    while (r > 1 && C1::kBaseBytes + (r - 1) * (C1::kStage + 16) > 232448) --r;
    r -= r % C1::kMaxSpl;
    return r;
}

// Fixed cost of finishing a segment, expressed as K+V bytes that could be
// streamed meanwhile, in pages of `heads` kv heads (rounded down);
// PA_SEG_WEIGHT_BYTES overrides it.
int32_t seg_weight_pages(int head_dim, int heads, int eb) {
    static const long long bytes = [] {
        const char* e = std::getenv("PA_SEG_WEIGHT_BYTES");
        return e ? std::atoll(e) : 65536LL;  // measured: 64 KB beats 32 KB on short contexts, equal on long
    }();
    const long long page = 2LL * kBlockSize * head_dim * eb * heads;
    return int32_t(bytes / page);
}

// kv heads per ring stage: as many whole K+V tiles (eb bytes per value) as a stage holds.
int heads_per_stage_max(int D, int eb, int stage_k) { return stage_k / (kBlockSize * D * eb); }

// kv heads per head group: the largest divisor of Hkv that is at most 8
// (one consumer warp per head) and splits into 1, 2, 4, ... max_spl equal stages.
int heads_per_group(int Hkv, int D, int eb, int stage_k, int max_spl) {
    const int hs = heads_per_stage_max(D, eb, stage_k);
    for (int h = pa::kDecodeWarps; h > 1; --h) {
        if (Hkv % h) continue;
        for (int spl = 1; spl <= max_spl; spl *= 2)
            if (h % spl == 0 && h / spl <= hs) return h;
    }
    return 1;
}

MathKind math_kind() {
    static const MathKind k = [] {
        const char* e = std::getenv("PA_DECODE_MATH");
        return (e && std::strcmp(e, "simt") == 0) ? MathKind::kSimt : MathKind::kMma;
    }();
    return k;
}

bool supported(int D, int G, MathKind mk) {
    if (D != 64 && D != 128) return false;
    if (G != 1 && G != 2 && G != 4 && G != 8) return false;
    return mk != MathKind::kSimt || G * D <= 256;
}

std::mutex g_mu;
int g_sms[kMaxDevices];

int current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    return dev;
}

int sm_count() {
    const int dev = current_device();
    if (dev < 0 || dev >= kMaxDevices) return -1;
    std::lock_guard<std::mutex> lock(g_mu);
    if (g_sms[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return -1;
        g_sms[dev] = n;
    }
    return g_sms[dev];
}

// Workspace layout: [counters: B*Hkv int32][part_o: grid*2*HG*G*D f32]
// [part_ml: grid*2*HG*G float2][group counters: grid*2*HG int32]
// [grid barrier of the fused append + decode: 2 uint32]
struct WsLayout {
    size_t counters, part_o, part_ml, slot_sync, grid_bar, total;
};

WsLayout ws_layout(const pa_dims& d, int grid) {
    // partial slots hold the query heads of one head group, at most min(Hkv, 8) kv heads (any cache format)
    const size_t hg_max = size_t(d.num_kv_heads < pa::kDecodeWarps ? d.num_kv_heads : pa::kDecodeWarps);
    const size_t hG = hg_max * (d.num_q_heads / d.num_kv_heads);
    WsLayout w;
    w.counters = 0;
    w.part_o = align_up(size_t(d.num_seqs) * d.num_kv_heads * 4, 256);
    w.part_ml = align_up(w.part_o + size_t(grid) * 2 * hG * d.head_dim * 4, 256);
    w.slot_sync = align_up(w.part_ml + size_t(grid) * 2 * hG * 8, 256);
    w.grid_bar = align_up(w.slot_sync + size_t(grid) * 2 * hg_max * 4, 256);
    w.total = w.grid_bar + 256;
    return w;
}

bool dims_ok(const pa_dims* d) {
    return d && d->num_seqs >= 0 && d->num_q_heads > 0 && d->num_kv_heads > 0 && d->head_dim > 0 &&
           d->block_size > 0 && d->num_blocks >= 0 && d->max_blocks_per_seq >= 0 &&
           d->num_q_heads % d->num_kv_heads == 0;
}

template <typename Kernel>
bool set_smem_once(Kernel kern, int bytes, unsigned* done_mask_per_device, bool wide_clusters = false) {
    const int dev = current_device();
    if (dev < 0 || dev >= kMaxDevices) return false;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!done_mask_per_device[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return false;
        // clusters of more than 8 CTAs
        if (wide_clusters && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return false;
        done_mask_per_device[dev] = 1;
    }
    return true;
}

#ifndef PA_L2_PROMOTION
#define PA_L2_PROMOTION CU_TENSOR_MAP_L2_PROMOTION_L2_256B
#endif

// cuTensorMapEncodeTiled from the driver, found through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// A cache [NB][Hkv][bs][D] bf16 seen as a 4-D tensor {64 columns, bs rows,
// D/64 panels, NB*Hkv tiles} (strides D*2 B, 128 B, bs*D*2 B).  One box is
// `heads` consecutive (block, kv head) tiles whole: {64, bs, D/64, heads},
// landing in shared memory as [tile][panel][row][128 B] with the 128-byte
// swizzle.
bool make_cache_map(CUtensorMap* map, const void* base, int64_t tiles, int D, int bs, int heads) {
    auto fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[4] = {64, cuuint64_t(bs), cuuint64_t(D / 64), cuuint64_t(tiles)};
    cuuint64_t strides[3] = {cuuint64_t(D) * 2, 128, cuuint64_t(bs) * D * 2};
    cuuint32_t box[4] = {64, cuuint32_t(bs), cuuint32_t(D / 64), cuuint32_t(heads)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, PA_L2_PROMOTION,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same 4-D view with a box of one 64-wide panel of one (block, kv head)
// tile: {64, 16, 1, 1} at {0, 0, panel, tile}, so a block of pages lands as
// [panel][tokens][128 bytes] (the tcgen05 operand layout).
bool make_panel_map(CUtensorMap* map, const void* base, int64_t tiles, int D, int bs) {
    auto fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[4] = {64, cuuint64_t(bs), cuuint64_t(D / 64), cuuint64_t(tiles)};
    cuuint64_t strides[3] = {cuuint64_t(D) * 2, 128, cuuint64_t(bs) * D * 2};
    cuuint32_t box[4] = {64, cuuint32_t(bs), 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, PA_L2_PROMOTION,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An fp8 cache seen as a 4-D uint8 tensor {128 bytes, D/8 lines, 1, NB*Hkv
// tiles} (rank 4 like the bf16 maps, so that the decode's 4-D tiled load
// {0, 0, 0, tile} serves both): one (block, kv head) tile is 16*D bytes =
// D/8 lines of 128 bytes (K: 16 tokens of D codes; V: D rows of 16 tokens).
// One box is `heads` consecutive tiles whole.  K takes the 128-byte swizzle
// (a line holds one token at head_dim 128, two at 64); V^T rows are 16
// bytes and need none.
bool make_fp8_map(CUtensorMap* map, const void* base, int64_t tiles, int D, int heads, bool swizzle) {
    auto fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[4] = {128, cuuint64_t(D / 8), 1, cuuint64_t(tiles)};
    cuuint64_t strides[3] = {128, cuuint64_t(16) * D, cuuint64_t(16) * D};
    cuuint32_t box[4] = {128, cuuint32_t(D / 8), 1, cuuint32_t(heads)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              PA_L2_PROMOTION, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// tcgen05 prefill configurations: BN keys per block, KS blocks in the ring,
// CPS CTAs per SM.
template <int D, int BN> constexpr int tc_stages() {
    return BN == 128 ? (D == 64 ? 4 : 3) : (D == 64 ? 5 : 2);
}

template <int D, int BN>
struct TcShape {
    static constexpr int KS = tc_stages<D, BN>(), CPS = BN == 128 ? 1 : 2;
    // S buffers: as many as TMEM holds next to O for CPS CTAs per SM
    static constexpr int NS = (3 * BN + D) * CPS <= 512 ? 3 : 2;
    using Cfg = pa::TcPrefillCfg<D, BN, KS, NS>;
    static_assert(CPS * (Cfg::kSmemBytes + 1024) <= 233472, "CTAs per SM by shared memory");
    static_assert(CPS * Cfg::kTmemCols <= 512, "CTAs per SM by TMEM columns");
};

// Shared validation of the decode calls; fills p.
pa_status prepare_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                         const int32_t* context_lens, float scale, void* out, const pa_dims* dims, int grid,
                         void* workspace, size_t workspace_bytes, pa::DecodeParams& p, int eb = 2,
                         MathKind mk = math_kind(), int stage_k = PA_STAGE_K_BYTES,
                         int max_spl = pa::kDecodeWarps) {
    if (!dims) return PA_ERR_NULL;
    if (!dims_ok(dims)) return PA_ERR_SHAPE;
    const pa_dims& d = *dims;
    const int G = d.num_q_heads / d.num_kv_heads;
    if (d.block_size != kBlockSize || !supported(d.head_dim, G, eb == 1 ? MathKind::kFp8 : mk))
        return PA_ERR_UNSUPPORTED;
    if (d.num_seqs == 0) return PA_OK;
    // at least one block, so that a bad block id can be redirected to block 0
    if (d.num_blocks == 0) return PA_ERR_SHAPE;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || !workspace) return PA_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(workspace) || !aligned4(block_tables) || !aligned4(context_lens))
        return PA_ERR_ALIGN;
    if (grid <= 0) return PA_ERR_CUDA;
    if (grid > kMaxCtas) return PA_ERR_SHAPE;
    const WsLayout w = ws_layout(d, grid);
    if (workspace_bytes < w.total) return PA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p = pa::DecodeParams{};
    const int64_t rows = int64_t(d.num_blocks) * d.num_kv_heads * d.block_size;
    if (rows >= (int64_t(1) << 31)) return PA_ERR_SHAPE;  // TMA coordinates are int32
    const int HG = heads_per_group(d.num_kv_heads, d.head_dim, eb, stage_k, max_spl);
    int SPL = 1;
    while (HG / SPL > heads_per_stage_max(d.head_dim, eb, stage_k) || HG % SPL) SPL *= 2;
    const int HS = HG / SPL;
    const int64_t tiles = int64_t(d.num_blocks) * d.num_kv_heads;
    const bool maps_ok =
        eb == 2 ? make_cache_map(&p.tmap_k, k_cache, tiles, d.head_dim, d.block_size, HS) &&
                      make_cache_map(&p.tmap_v, v_cache, tiles, d.head_dim, d.block_size, HS)
                : make_fp8_map(&p.tmap_k, k_cache, tiles, d.head_dim, HS, true) &&
                      make_fp8_map(&p.tmap_v, v_cache, tiles, d.head_dim, HS, false);
    if (!maps_ok) return PA_ERR_CUDA;
    p.q = static_cast<const uint8_t*>(q);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.qscale = scale * kLog2e;
    p.B = d.num_seqs;
    p.Hq = d.num_q_heads;
    p.Hkv = d.num_kv_heads;
    p.NB = d.num_blocks;
    p.M = d.max_blocks_per_seq;
    p.HG = HG;
    p.NG = d.num_kv_heads / HG;
    p.HS = HS;
    p.SPL = SPL;
    p.SPL_LOG = SPL == 1 ? 0 : SPL == 2 ? 1 : SPL == 4 ? 2 : 3;
    p.min_pages = kMinPagesPerCta;
    p.seg_weight = seg_weight_pages(d.head_dim, HG, eb);
    p.counters = reinterpret_cast<int32_t*>(ws + w.counters);
    p.part_o = reinterpret_cast<float*>(ws + w.part_o);
    p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
    p.slot_sync = reinterpret_cast<int32_t*>(ws + w.slot_sync);
    p.grid_bar = reinterpret_cast<unsigned int*>(ws + w.grid_bar);
    return PA_OK;
}

}  // namespace
