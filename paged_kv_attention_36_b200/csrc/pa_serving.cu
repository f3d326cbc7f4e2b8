// pa_serving.cu -- the entry points of include/pa.h for windowed attention,
// the 8-bit cache with a scale for each (block, kv head), and the append with
// the position rotation: host-side checks and launches.
#include <atomic>

#include <type_traits>

#include "pa_cluster.cuh"
#include "pa_decode_wide.cuh"
#include "pa_host.cuh"
#include "pa_prefill_i8.cuh"
#include "pa_rope.cuh"

bool pa::serving_error_word(unsigned int* bits, bool clear) { return read_error_word(bits, clear); }

namespace {

pa_status launched() { return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

struct Call {  // the arguments the attention calls share
    const void* q;
    const int32_t* cu_q_lens;
    int32_t max_q_len;
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;
    const float* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    float scale;
    int32_t window, sinks;
    void* out;
    const pa_dims* dims;
};

bool window_ok(int32_t window, int32_t sinks) { return window >= 1 && sinks >= 0; }

pa_status scales_ok(const Call& c) {
    if (!c.k_scale || !c.v_scale) return PA_ERR_NULL;
    return aligned4(c.k_scale) && aligned4(c.v_scale) ? PA_OK : PA_ERR_ALIGN;
}

// Checks of a multi-query call; *done: there is nothing to compute.
pa_status check_prefill(const Call& c, bool* done) {
    *done = true;
    if (!c.dims) return PA_ERR_NULL;
    if (!dims_ok(c.dims) || c.max_q_len < 0 || !window_ok(c.window, c.sinks)) return PA_ERR_SHAPE;
    const pa_dims& d = *c.dims;
    const int G = d.num_q_heads / d.num_kv_heads;
    if (d.block_size != kBlockSize || !supported(d.head_dim, G, MathKind::kMma)) return PA_ERR_UNSUPPORTED;
    if (d.num_seqs == 0 || c.max_q_len == 0) return PA_OK;
    if (d.num_blocks == 0) return PA_ERR_SHAPE;
    if (!c.q || !c.cu_q_lens || !c.k_cache || !c.v_cache || !c.block_tables || !c.context_lens || !c.out)
        return PA_ERR_NULL;
    if (!aligned16(c.q) || !aligned16(c.out) || !aligned16(c.k_cache) || !aligned16(c.v_cache) ||
        !aligned4(c.cu_q_lens) || !aligned4(c.block_tables) || !aligned4(c.context_lens))
        return PA_ERR_ALIGN;
    if (int64_t(d.num_blocks) * d.num_kv_heads * d.block_size >= (int64_t(1) << 31)) return PA_ERR_SHAPE;
    const int64_t tiles = (int64_t(c.max_q_len) * G + 127) / 128;
    if (tiles > 0x7fffffffLL || int64_t(d.num_seqs) * tiles > 0x7fffffffLL / d.num_kv_heads) return PA_ERR_SHAPE;
    *done = false;
    return PA_OK;
}

void fill_prefill(const Call& c, pa::PrefillParams& p) {
    const pa_dims& d = *c.dims;
    p.q = static_cast<const uint8_t*>(c.q);
    p.cu_q_lens = c.cu_q_lens;
    p.block_tables = c.block_tables;
    p.context_lens = c.context_lens;
    p.out = static_cast<__nv_bfloat16*>(c.out);
    p.B = d.num_seqs;
    p.Hq = d.num_q_heads;
    p.Hkv = d.num_kv_heads;
    p.NB = d.num_blocks;
    p.M = d.max_blocks_per_seq;
    p.tiles_per_seq = int32_t((int64_t(c.max_q_len) * (d.num_q_heads / d.num_kv_heads) + 127) / 128);
    p.qscale = c.scale * kLog2e;
    p.window = c.window;
    p.sinks = c.sinks;
    p.v_cache = static_cast<const uint8_t*>(c.v_cache);
}

// fn<D, G>() for the head_dim and GQA group of a call that supported() let through.
template <class F>
pa_status by_shape(const pa_dims& d, F fn) {
    const int G = d.num_q_heads / d.num_kv_heads;
    auto with = [&](auto dim) -> pa_status {
        constexpr int D = decltype(dim)::value;
        switch (G) {
            case 1: return fn.template operator()<D, 1>();
            case 2: return fn.template operator()<D, 2>();
            case 4: return fn.template operator()<D, 4>();
            case 8: return fn.template operator()<D, 8>();
        }
        return PA_ERR_UNSUPPORTED;
    };
    return d.head_dim == 64 ? with(std::integral_constant<int, 64>{}) : with(std::integral_constant<int, 128>{});
}

// Launches with programmatic serialization: the kernel's set-up may overlap
// the end of the one before it (it waits with griddepcontrol.wait).
// `cluster` CTAs (along x) form a cluster.
template <class Kernel, class Params>
pa_status launch_dependent(Kernel kern, dim3 grid, int threads, int smem, cudaStream_t stream, const Params& p,
                           unsigned cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return PA_ERR_CUDA;
    return launched();
}

// ---- wide decode ---------------------------------------------------------------
constexpr int kWideStageK = 8192;      // K bytes of a ring stage, at most (windowed batch: 48.0 us, 49.5 us at 16 KB)
// K+V bytes worth a CTA of their own (4 short sequences: 5.4 us; 8.1 us at
// 4 KB, where contexts are cut and merged, 7.3 us at 256 KB, where CTAs queue
// them; a batch of 128 does not notice)
constexpr int kWideMinBytes = 65536;
constexpr int kMaxSmem = 232448;

int floor_log2(int x) {
    int n = 0;
    while (x >> (n + 1)) ++n;
    return n;
}

// The ring and the warps for p's head layout; false if it cannot be (no supported layout).
bool wide_shape(const pa::DecodeParams& p, int D, int eb, pa::WideShape& s) {
    const int tile = kBlockSize * D * eb;
    s.HG = p.HG;
    s.HS = p.HS;
    s.SPL_LOG = p.SPL_LOG;
    s.WPH_LOG = floor_log2(pa::kWideWarps / p.HG);
    s.stage_k = p.HS * tile;
    const int step = 1 << (s.SPL_LOG + s.WPH_LOG);
    for (s.R = pa::kWideMaxRing / step * step; s.R > 0; s.R -= step)
        if (pa::wide_layout(s, D).total + 1024 <= kMaxSmem) break;
    s.smem = pa::wide_layout(s, D).total + 1024;
    return s.R > 0;
}

template <bool I8>
struct DecodeWide {
    pa::WideParams& p;
    int grid;
    cudaStream_t stream;
    template <int D, int G>
    pa_status operator()() const {
        using MathT = std::conditional_t<I8, pa::I8Math<D, G>, pa::MmaMath<D, G, kBlockSize>>;
        auto kern = pa::decode_wide_kernel<MathT, D, G, I8>;
        static unsigned attr_done[kMaxDevices];
        if (!set_smem_once(kern, kMaxSmem, attr_done)) return PA_ERR_CUDA;
        if (!wide_shape(p.d, D, I8 ? 1 : 2, p.shape)) return PA_ERR_UNSUPPORTED;
        const int page = 2 * kBlockSize * D * (I8 ? 1 : 2) * p.d.HG;
        p.d.min_pages = kWideMinBytes / page > 2 ? kWideMinBytes / page : 2;
        p.shape.snap = p.d.min_pages / 2;
        return launch_dependent(kern, dim3(unsigned(grid)), pa::kWideThreads, p.shape.smem, stream, p);
    }
};

template <bool I8>
pa_status decode_wide(const Call& c, void* workspace, size_t workspace_bytes, void* stream) {
    if (!c.dims) return PA_ERR_NULL;
    if (!window_ok(c.window, c.sinks)) return PA_ERR_SHAPE;
    pa::WideParams p;
    const int grid = sm_count();
    pa_status st = prepare_decode(c.q, c.k_cache, c.v_cache, c.block_tables, c.context_lens, c.scale, c.out, c.dims,
                                  grid, workspace, workspace_bytes, p.d, I8 ? 1 : 2, MathKind::kMma, kWideStageK,
                                  /*max_spl=*/1);
    if (st != PA_OK || c.dims->num_seqs == 0) return st;
    if (I8 && (st = scales_ok(c)) != PA_OK) return st;
    p.d.k_scale = c.k_scale;
    p.d.v_scale = c.v_scale;
    p.window = c.window;
    p.sinks = c.sinks;
    return by_shape(*c.dims, DecodeWide<I8>{p, grid, static_cast<cudaStream_t>(stream)});
}

// Key blocks of the longest row that the tables and the window allow.
int64_t key_blocks(const Call& c) {
    int64_t keys = int64_t(c.dims->max_blocks_per_seq) * kBlockSize;
    const int64_t seen = int64_t(c.window) + c.sinks + c.max_q_len;
    if (seen < keys) keys = seen;
    return (keys + 63) / 64;
}

constexpr int kAloneSmem = 122880;  // shared memory that leaves a CTA its SM to itself

// Clusters of n CTAs of a kernel that the current device holds at once; asked once
// per kernel, size and device (`cache`, 0: not asked yet, -1: none).
using HeldCache = std::atomic<int>[kMaxDevices * 16];
template <class Kernel>
int clusters_held(Kernel kern, int threads, int smem, unsigned n, bool alone, HeldCache& cache) {
    std::atomic<int>& held = cache[(current_device() * 8 + floor_log2(int(n))) * 2 + alone];
    int count = held.load(std::memory_order_relaxed);
    if (count == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n);
        cfg.blockDim = dim3(unsigned(threads));
        cfg.dynamicSmemBytes = size_t(alone ? kAloneSmem : smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = n;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&count, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            count = 0;
        }
        if (count <= 0) count = -1;
        held.store(count, std::memory_order_relaxed);
    }
    return count > 0 ? count : 0;
}

// Launches `whole`, a kernel with a CTA a tile, or `split`, with a cluster a tile.
template <class Kernel, class Params>
pa_status launch_tiles(Kernel whole, Kernel split, int threads, int smem, unsigned tiles, int64_t blocks, int sms,
                       unsigned* whole_done, unsigned* split_done, HeldCache& cache, cudaStream_t stream,
                       const Params& p) {
    if (pa::wanted_ranks(tiles, blocks, sms) > 1) {
        if (!set_smem_once(split, kAloneSmem, split_done, true)) return PA_ERR_CUDA;
        const pa::ClusterChoice c = pa::choose_cluster(tiles, blocks, sms, [&](unsigned n, bool alone) -> int64_t {
            return clusters_held(split, threads, smem, n, alone, cache);
        });
        if (c.ranks > 1)
            return launch_dependent(split, dim3(tiles * c.ranks), threads, c.alone ? kAloneSmem : smem, stream, p,
                                    c.ranks);
    }
    if (!set_smem_once(whole, smem, whole_done)) return PA_ERR_CUDA;
    return launch_dependent(whole, dim3(tiles), threads, smem, stream, p);
}

struct PrefillWindow {
    const pa::PrefillParams& p;
    unsigned tiles;
    int64_t blocks;
    int sms;
    cudaStream_t stream;
    template <int D, int G>
    pa_status operator()() const {
        using S = TcShape<D, 64>;
        static_assert(S::Cfg::kWindowSmemBytes <= kAloneSmem);
        static unsigned done[2][kMaxDevices];
        static HeldCache held;
        return launch_tiles(pa::prefill_tc_kernel<D, G, 64, S::KS, S::CPS, S::NS, true, false>,
                            pa::prefill_tc_kernel<D, G, 64, S::KS, S::CPS, S::NS, true, true>, S::Cfg::kThreads,
                            S::Cfg::kWindowSmemBytes, tiles, blocks, sms, done[0], done[1], held, stream, p);
    }
};

struct PrefillI8 {
    const pa::PrefillI8Params& p;
    unsigned tiles;
    int64_t blocks;
    int sms;
    cudaStream_t stream;
    template <int D, int G>
    pa_status operator()() const {
        using Cfg = pa::I8PrefillCfg<D>;
        static_assert(Cfg::kSmemBytes <= kAloneSmem);
        const auto whole = pa::prefill_i8_kernel<D, G, false>, split = pa::prefill_i8_kernel<D, G, true>;
        // the kernels' setmaxnreg split needs exactly the registers it counts on
        static const bool regs_ok = [&] {
            cudaFuncAttributes a, b;
            return cudaFuncGetAttributes(&a, whole) == cudaSuccess && a.numRegs == Cfg::kRegs &&
                   cudaFuncGetAttributes(&b, split) == cudaSuccess && b.numRegs == Cfg::kRegs;
        }();
        if (!regs_ok) return PA_ERR_CUDA;
        static unsigned done[2][kMaxDevices];
        static HeldCache held;
        return launch_tiles(whole, split, Cfg::kThreads, Cfg::kSmemBytes, tiles, blocks, sms, done[0], done[1], held,
                            stream, p);
    }
};

struct Append {  // the arguments of an append with rotation
    const void* q;
    int64_t q_stride;
    const void* k_new;
    int64_t k_stride;
    const void* v_new;
    int64_t v_stride;
    const pa_rope* rope;
    const int32_t* slot_mapping;
    int32_t num_tokens;
    void* q_out;
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    const pa_dims* dims;
};

// Checks an append and fills p; p.T = 0: there is nothing to do.
pa_status prepare_append(const Append& a, bool i8, pa::RopeParams& p) {
    p = pa::RopeParams{};
    if (!a.dims) return PA_ERR_NULL;
    const pa_dims& d = *a.dims;
    const int rd = a.rope ? a.rope->rotary_dim : 0;
    if (a.num_tokens < 0 || d.num_kv_heads <= 0 || d.head_dim <= 0 || d.block_size <= 0 || d.num_blocks < 0 ||
        (a.q && d.num_q_heads <= 0) || rd < 0 || rd > d.head_dim)
        return PA_ERR_SHAPE;
    if (d.head_dim % 16 != 0 || rd % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (i8 && (d.block_size != kBlockSize || (d.head_dim != 64 && d.head_dim != 128))) return PA_ERR_UNSUPPORTED;
    if (a.num_tokens == 0) return PA_OK;
    if (!a.k_new || !a.v_new || !a.slot_mapping || !a.k_cache || !a.v_cache || (a.q && !a.q_out) ||
        (i8 && (!a.k_scale || !a.v_scale)))
        return PA_ERR_NULL;
    if (rd > 0) {
        if (!a.rope->positions || !a.rope->cos_sin) return PA_ERR_NULL;
        if (a.rope->max_position <= 0) return PA_ERR_SHAPE;
        if (!aligned4(a.rope->positions) || !aligned16(a.rope->cos_sin)) return PA_ERR_ALIGN;
    }
    const int64_t qw = int64_t(d.num_q_heads) * d.head_dim, kw = int64_t(d.num_kv_heads) * d.head_dim;
    if ((a.q && a.q_stride < qw) || a.k_stride < kw || a.v_stride < kw) return PA_ERR_SHAPE;
    if ((a.q && a.q_stride % 8) || a.k_stride % 8 || a.v_stride % 8 || (a.q && (!aligned16(a.q) || !aligned16(a.q_out))) ||
        !aligned16(a.k_new) || !aligned16(a.v_new) || !aligned16(a.k_cache) || !aligned16(a.v_cache) ||
        !aligned4(a.slot_mapping) || (i8 && (!aligned4(a.k_scale) || !aligned4(a.v_scale))))
        return PA_ERR_ALIGN;
    if (a.q && !(a.q == a.q_out && a.q_stride == qw)) {  // in place, or apart: rows written before they are read otherwise
        const uintptr_t q0 = reinterpret_cast<uintptr_t>(a.q), o0 = reinterpret_cast<uintptr_t>(a.q_out);
        const uintptr_t q1 = q0 + ((a.num_tokens - 1) * a.q_stride + qw) * 2, o1 = o0 + a.num_tokens * qw * 2;
        // q's rows may lie between rows of another buffer, q_out's do not
        if (q0 < o1 && o0 < q1) return PA_ERR_SHAPE;
    }
    if (int64_t(d.num_blocks) * d.block_size > 0x7fffffffLL) return PA_ERR_SHAPE;  // slots are int32
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k_new = static_cast<const __nv_bfloat16*>(a.k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(a.v_new);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    if (rd > 0) {
        p.positions = a.rope->positions;
        p.cos_sin = a.rope->cos_sin;
        p.max_position = a.rope->max_position;
        p.interleaved = a.rope->interleaved != 0;
    }
    p.rd = rd;
    p.slot_mapping = a.slot_mapping;
    p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.T = a.num_tokens;
    p.Hq = a.q ? d.num_q_heads : 0;
    p.Hkv = d.num_kv_heads;
    p.D = d.head_dim;
    p.bs = d.block_size;
    p.NB = d.num_blocks;
    return PA_OK;
}

// Rows a thread takes: four share one read of the angles once there are enough
// threads for every SM without (2048 each): 8192 tokens 37.8 us against 41.6 us
// a row each; a step of 128 tokens 3.7 us a row each, 3.9 us in fours.
bool rows_in_fours(int64_t rows, int D, int sms) { return rows * (D / 16) >= int64_t(4) * 2048 * sms; }

template <int HP>
pa_status launch_rope(const pa::RopeParams& p, cudaStream_t s) {
    const int64_t items = int64_t(p.T) * ((p.Hq + 2 * p.Hkv + HP - 1) / HP) * (p.D / 16);
    if (items >= int64_t(1) << 32) return PA_ERR_SHAPE;
    const unsigned ctas = unsigned((items + pa::kRopeThreads - 1) / pa::kRopeThreads);
    return launch_dependent(pa::rope_append_kernel<HP>, dim3(ctas), pa::kRopeThreads, 0, s, p);
}

template <int D, int HP>
pa_status launch_rope_i8(pa::RopeParams& p, int sms, cudaStream_t s) {
    const int64_t items = int64_t(p.T) * ((p.Hq + HP - 1) / HP) * (D / 16);
    if (items >= int64_t(1) << 32) return PA_ERR_SHAPE;
    // a decode step's tokens have a block each and a CTA each (128 tokens: 4.9 us,
    // 31.9 us with 16 to a CTA); of a long call's tokens few are their block's
    // first, and a CTA looks at up to 16 (7295 tokens: 56.7 us, 59.4 us with one)
    p.tokens_per_cta = p.T <= 4 * sms ? 1 : p.T / (4 * sms) < 16 ? p.T / (4 * sms) : 16;
    // a tile per warp: as many CTAs as a block's tiles need, while there are SMs
    // for them (128 tokens, 8 kv heads: 4.9 us, 6.6 us with two tiles a warp)
    const int groups = (p.T + p.tokens_per_cta - 1) / p.tokens_per_cta, warps = pa::kRopeThreads / 32;
    p.parts = (2 * p.Hkv + warps - 1) / warps;
    while (p.parts > 1 && int64_t(groups) * p.parts > 12 * sms) --p.parts;
    p.kv_ctas = groups * p.parts;
    const int64_t ctas = p.kv_ctas + (items + pa::kRopeThreads - 1) / pa::kRopeThreads;
    if (ctas > 0x7fffffff) return PA_ERR_SHAPE;
    constexpr int smem = 16 * D * 4 + pa::kRopeThreads / 32 * 16 * D * 2;  // angles, a tile a warp
    static unsigned attr_done[kMaxDevices];
    if (!set_smem_once(pa::rope_append_i8_kernel<D, HP>, smem, attr_done)) return PA_ERR_CUDA;
    return launch_dependent(pa::rope_append_i8_kernel<D, HP>, dim3(unsigned(ctas)), pa::kRopeThreads, smem, s, p);
}

pa_status append_i8(const Append& a, cudaStream_t s) {
    pa::RopeParams p;
    const pa_status st = prepare_append(a, true, p);
    if (st != PA_OK || p.T == 0) return st;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const bool many = rows_in_fours(int64_t(p.T) * p.Hq, p.D, sms);  // in twos here: four leave too few registers
    if (p.D == 64) return many ? launch_rope_i8<64, 2>(p, sms, s) : launch_rope_i8<64, 1>(p, sms, s);
    return many ? launch_rope_i8<128, 2>(p, sms, s) : launch_rope_i8<128, 1>(p, sms, s);
}

}  // namespace

extern "C" {

pa_status pa_decode_window(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                           const int32_t* context_lens, float scale, int32_t window, int32_t sinks, void* out,
                           const pa_dims* dims, void* workspace, size_t workspace_bytes, void* stream) {
    const Call c{q, nullptr, 1, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, scale, window, sinks,
                 out, dims};
    return decode_wide<false>(c, workspace, workspace_bytes, stream);
}

pa_status pa_decode_i8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, const int32_t* block_tables, const int32_t* context_lens, float scale,
                       int32_t window, int32_t sinks, void* out, const pa_dims* dims, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const Call c{q, nullptr, 1, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, window, sinks,
                 out, dims};
    return decode_wide<true>(c, workspace, workspace_bytes, stream);
}

pa_status pa_prefill_window(const void* q, const int32_t* cu_q_lens, int32_t max_q_len, const void* k_cache,
                            const void* v_cache, const int32_t* block_tables, const int32_t* context_lens, float scale,
                            int32_t window, int32_t sinks, void* out, const pa_dims* dims, void* stream) {
    const Call c{q, cu_q_lens, max_q_len, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, scale,
                 window, sinks, out, dims};
    bool done;
    const pa_status st = check_prefill(c, &done);
    if (st != PA_OK || done) return st;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const pa_dims& d = *dims;
    pa::PrefillParams p;
    const int64_t cache_tiles = int64_t(d.num_blocks) * d.num_kv_heads;
    if (!make_panel_map(&p.tmap_k, k_cache, cache_tiles, d.head_dim, d.block_size) ||
        !make_panel_map(&p.tmap_v, v_cache, cache_tiles, d.head_dim, d.block_size))
        return PA_ERR_CUDA;
    fill_prefill(c, p);
    const unsigned tiles = unsigned(d.num_seqs * p.tiles_per_seq * d.num_kv_heads);
    return by_shape(d, PrefillWindow{p, tiles, key_blocks(c), sms, static_cast<cudaStream_t>(stream)});
}

pa_status pa_prefill_i8(const void* q, const int32_t* cu_q_lens, int32_t max_q_len, const void* k_cache,
                        const void* v_cache, const float* k_scale, const float* v_scale, const int32_t* block_tables,
                        const int32_t* context_lens, float scale, int32_t window, int32_t sinks, void* out,
                        const pa_dims* dims, void* stream) {
    const Call c{q, cu_q_lens, max_q_len, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                 window, sinks, out, dims};
    bool done;
    pa_status st = check_prefill(c, &done);
    if (st != PA_OK || done) return st;
    if ((st = scales_ok(c)) != PA_OK) return st;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    pa::PrefillI8Params p{};
    fill_prefill(c, p.a);
    p.k_cache = static_cast<const int8_t*>(k_cache);
    p.v_cache = static_cast<const int8_t*>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    const unsigned tiles = unsigned(dims->num_seqs * p.a.tiles_per_seq * dims->num_kv_heads);
    return by_shape(*dims, PrefillI8{p, tiles, key_blocks(c), sms, static_cast<cudaStream_t>(stream)});
}

pa_status pa_rope_append(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                         int64_t v_stride, const pa_rope* rope, const int32_t* slot_mapping, int32_t num_tokens,
                         void* q_out, void* k_cache, void* v_cache, const pa_dims* dims, void* stream) {
    pa::RopeParams p;
    const pa_status st = prepare_append(Append{q, q_stride, k_new, k_stride, v_new, v_stride, rope, slot_mapping,
                                               num_tokens, q_out, k_cache, v_cache, nullptr, nullptr, dims},
                                        false, p);
    if (st != PA_OK || p.T == 0) return st;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return rows_in_fours(int64_t(p.T) * (p.Hq + 2 * p.Hkv), p.D, sms) ? launch_rope<4>(p, s) : launch_rope<1>(p, s);
}

pa_status pa_rope_append_i8(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                            int64_t v_stride, const pa_rope* rope, const int32_t* slot_mapping, int32_t num_tokens,
                            void* q_out, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                            const pa_dims* dims, void* stream) {
    return append_i8(Append{q, q_stride, k_new, k_stride, v_new, v_stride, rope, slot_mapping, num_tokens, q_out,
                            k_cache, v_cache, k_scale, v_scale, dims},
                     static_cast<cudaStream_t>(stream));
}

pa_status pa_cache_append_i8(const void* k_new, const void* v_new, const int32_t* slot_mapping, int32_t num_tokens,
                             void* k_cache, void* v_cache, float* k_scale, float* v_scale, const pa_dims* dims,
                             void* stream) {
    if (!dims) return PA_ERR_NULL;
    const int64_t w = int64_t(dims->num_kv_heads) * dims->head_dim;
    return append_i8(Append{nullptr, 0, k_new, w, v_new, w, nullptr, slot_mapping, num_tokens, nullptr, k_cache,
                            v_cache, k_scale, v_scale, dims},
                     static_cast<cudaStream_t>(stream));
}

}  // extern "C"
