// pa_decode_wide.cuh -- paged decode with a sliding window, and over 8-bit
// caches with a scale for each (block, kv head).
//
// The work line, the ring of TMA-staged pages, the split-KV partials and
// their merge are those of pa_decode.cuh.  What differs:
//
//   * Several warps share a kv head.  A CTA has 16 consumer warps, WPH = the
//     largest power of two <= 16 / HG of them per head of the head group;
//     part w of a head takes the pages whose running number is w modulo WPH
//     and keeps a softmax state of its own.  At a segment's end the parts
//     meet in shared memory and part 0 finishes the segment while the others
//     go on.  The page math is a dependent chain (ldmatrix, convert, mma,
//     max, exp2, mma), so one warp per head leaves the SM's issue slots
//     empty: at half the bytes per token that chain, not HBM, was the bound
//     of the fp8 decode (one warp per head: 34 % issue, 55 % DRAM).
//   * Only the pages that a window or a sink reaches are on the line
//     (WindowPages), and each page comes with a 16-bit mask of the tokens
//     that count.
//   * Share boundaries that would cut fewer than `snap` pages off a segment
//     move to the segment's end (cut_page): short contexts stay whole, so a
//     small batch needs no merge between CTAs.
//   * A page of an 8-bit cache brings its heads' scales along: 4-byte
//     cp.async copies that arrive on the stage's barrier.
//   * Launched as a programmatic dependent: the set-up overlaps the end of
//     the kernel before it.
#pragma once

#include "pa_decode.cuh"

namespace pa {

// Page at which a share boundary at line position t cuts a segment of np
// pages that starts at u0: 0 or np where fewer than `snap` pages (or half
// the segment) would lie before or behind it.
__host__ __device__ __forceinline__ int32_t cut_page(int64_t t, int64_t u0, int32_t np, int32_t snap) {
    if (t <= u0) return 0;
    if (t >= u0 + np) return np;
    const int32_t c = int32_t(t - u0), lo = snap < (np + 1) / 2 ? snap : (np + 1) / 2;
    return c < lo ? 0 : np - c < lo ? np : c;
}

// ---- page math over 8-bit codes ------------------------------------------------
// The tiles are the fp8 policy's (K [16][D] in 128-byte swizzled lines, V
// transposed in its token order), so the fragments are too: plain ldmatrix
// gives a lane four consecutive codes of a row.  A code b becomes an f16 by
// its bytes alone: 0x6400 | (b ^ 0x80) is 1024 + 128 + b.  For K the 1152 is
// taken back at once for the whole dot product (the accumulator starts at
// -1152 sum(q)); for V, whose sums are long, value by value (exact).  Queries
// are scaled by a power of two to at most 2 in f16, which loses nothing
// bf16 holds down to 2^-14 of the row's largest value; P goes into the second
// product as f16 (2^-11).  Each page's P V is scaled by the page's V scale
// when it is added to the fp32 state.
template <int D, int G>
struct I8Math : MmaMath<D, G, 16> {
    using Base = MmaMath<D, G, 16>;
    using Base::KS;
    using Base::qb;
    using Base::acc;
    using Base::m;
    using Base::l;
    static constexpr int kElemBytes = 1;
    float qs[2];    // scale * log2(e) * the query's power of two, heads h0 and h0 + 1
    float bias[2];  // -1152 * sum of the query's f16 values

    __device__ __forceinline__ void load_q_global(const uint8_t* gq, int lane, float qscale) {
        const int h = lane >> 2, c = lane & 3;
        uint2 w[KS];
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            w[ks] = h < G ? __ldg(reinterpret_cast<const uint2*>(gq + (h * D + 16 * ks + 4 * c) * 2)) : make_uint2(0, 0);
            const float2 a = bf16x2_to_float2(w[ks].x), b = bf16x2_to_float2(w[ks].y);
            top = fmaxf(fmaxf(top, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = top > 0.f && top < INFINITY ? ilogbf(top) : 0;
        const float down = exp2f(float(-e));
        float sum = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const float2 a = bf16x2_to_float2(w[ks].x), b = bf16x2_to_float2(w[ks].y);
            qb[ks][0] = float2_to_f16x2(a.x * down, a.y * down);
            qb[ks][1] = float2_to_f16x2(b.x * down, b.y * down);
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&qb[ks][0]));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&qb[ks][1]));
            sum += (x.x + x.y) + (y.x + y.y);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const float up = qscale * exp2f(float(e));
        // a lane's logits are heads h0, h0 + 1, whose rows lanes 4 h0 .. hold
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int from = 4 * (2 * c + i);
            qs[i] = __shfl_sync(0xffffffffu, up, from);
            bias[i] = -1152.f * __shfl_sync(0xffffffffu, sum, from);
        }
    }

    // Byte offset of 16-byte chunk ch (d 16ch .. 16ch+15) of token t in a K tile.
    static __device__ __forceinline__ int k_off(int t, int ch) {
        const int line = D == 128 ? t : (t >> 1);
        const int lch = D == 128 ? ch : (((t & 1) << 2) + ch);
        return (line << 7) + ((lch ^ (line & 7)) << 4);
    }
    // Codes (0, 1) and (2, 3) of four, plus 1152, as f16 pairs.
    static __device__ __forceinline__ void biased(uint32_t r, uint32_t& lo, uint32_t& hi) {
        r ^= 0x80808080u;
        lo = __byte_perm(r, 0x64646464u, 0x4140);
        hi = __byte_perm(r, 0x64646464u, 0x4342);
    }
    static __device__ __forceinline__ void codes(uint32_t r, uint32_t& lo, uint32_t& hi) {
        biased(r, lo, hi);
        const __half2 b = __floats2half2_rn(1152.f, 1152.f);
        __half2 x = __hsub2(*reinterpret_cast<__half2*>(&lo), b), y = __hsub2(*reinterpret_cast<__half2*>(&hi), b);
        lo = *reinterpret_cast<uint32_t*>(&x);
        hi = *reinterpret_cast<uint32_t*>(&y);
    }

    __device__ __forceinline__ void page(const uint8_t* kt, const uint8_t* vt, uint32_t vis, float ks, float vs,
                                         int lane) {
        const int mi = lane >> 3, r8 = lane & 7;
        // ---- S^T = K . Q^T ----
        float s[4] = {bias[0], bias[1], bias[0], bias[1]};
        {
            const int t = r8 + ((mi & 1) << 3);
#pragma unroll
            for (int j = 0; j < KS / 2; ++j) {
                uint32_t r[4], a0[4], a1[4];
                ldmatrix_x4(r, kt + k_off(t, 2 * j + (mi >> 1)));
                biased(r[0], a0[0], a0[2]);
                biased(r[1], a0[1], a0[3]);
                biased(r[2], a1[0], a1[2]);
                biased(r[3], a1[1], a1[3]);
                mma_f16_16816(s, a0, qb[2 * j][0], qb[2 * j][1]);
                mma_f16_16816(s, a1, qb[2 * j + 1][0], qb[2 * j + 1][1]);
            }
        }
        const int t0 = lane >> 2;
        const bool v0 = (vis >> t0) & 1, v1 = (vis >> (t0 + 8)) & 1;
        const float c0 = qs[0] * ks, c1 = qs[1] * ks;
        s[0] = v0 ? s[0] * c0 : -INFINITY;
        s[1] = v0 ? s[1] * c1 : -INFINITY;
        s[2] = v1 ? s[2] * c0 : -INFINITY;
        s[3] = v1 ? s[3] * c1 : -INFINITY;
        // ---- online softmax over the 16 tokens of each head column ----
        float mx0 = fmaxf(s[0], s[2]), mx1 = fmaxf(s[1], s[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
        }
        if (__any_sync(0xffffffffu, mx0 > m[0] || mx1 > m[1])) {
            const float n0 = fmaxf(m[0], mx0), n1 = fmaxf(m[1], mx1);
            this->rescale(exp2f(m[0] - n0), exp2f(m[1] - n1));
            m[0] = n0;
            m[1] = n1;
        }
        const float p0 = exp2f(s[0] - m[0]), p1 = exp2f(s[1] - m[1]);
        const float p2 = exp2f(s[2] - m[0]), p3 = exp2f(s[3] - m[1]);
        l[0] += p0 + p2;
        l[1] += p1 + p3;
        // ---- O^T += v_scale * V^T . P^T, two m-tiles (32 rows of V^T) per ldmatrix ----
        const uint32_t b0 = movmatrix_trans(float2_to_f16x2(p0, p1));
        const uint32_t b1 = movmatrix_trans(float2_to_f16x2(p2, p3));
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            uint32_t r[4], a0[4], a1[4];
            ldmatrix_x4(r, vt + (32 * j + lane) * 16);
            codes(r[0], a0[0], a0[2]);
            codes(r[1], a0[1], a0[3]);
            codes(r[2], a1[0], a1[2]);
            codes(r[3], a1[1], a1[3]);
            float o0[4] = {0.f, 0.f, 0.f, 0.f}, o1[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16_16816(o0, a0, b0, b1);
            mma_f16_16816(o1, a1, b0, b1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * j][i] += vs * o0[i];
                acc[2 * j + 1][i] += vs * o1[i];
            }
        }
    }

    __device__ __forceinline__ void rescale(float a0, float a1) {
        l[0] *= a0;
        l[1] *= a1;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            acc[i][0] *= a0;
            acc[i][1] *= a1;
            acc[i][2] *= a0;
            acc[i][3] *= a1;
        }
    }
};

// ---- shared memory ---------------------------------------------------------------
constexpr int kWideWarps = 16;  // consumer warps
constexpr int kWideThreads = (kWideWarps + 1) * 32;
constexpr int kWideSegs = 4;    // segment descriptors in flight
constexpr int kWideMaxRing = 32;

// How a call's head layout uses the CTA (computed on the host).
struct WideShape {
    int32_t HG, HS, SPL_LOG, WPH_LOG;  // heads per group and per stage, log2 of stages per page and of warps per head
    int32_t R;                         // ring stages, a multiple of (stages per page) * (warps per head)
    int32_t stage_k;                   // K bytes of a stage (as many V bytes follow)
    int32_t snap;                      // fewest pages worth cutting off a segment
    int32_t smem;                      // bytes
};

struct WideLayout {  // byte offsets from the 1024-byte aligned base
    int32_t ring, parts, scales, descs, bars, misc, total;
};

// A part's state in shared memory: the accumulator fragments as they lie in
// the lanes, then (m, l) of the lane's two heads.
__host__ __device__ constexpr int part_bytes(int D) { return (D / 16 + 1) * 32 * 16; }

struct WideMisc {
    int abort;
    int b0, L0;         // sequence where the share starts, its length
    long long pre0;     // line position of its first unit
    long long red[kWideWarps + 1];
};

__host__ __device__ inline WideLayout wide_layout(const WideShape& s, int D) {
    WideLayout w;
    const int wph = 1 << s.WPH_LOG;
    w.ring = 0;
    w.parts = s.R * 2 * s.stage_k;
    w.scales = w.parts + (wph - 1) * s.HG * part_bytes(D);
    w.descs = w.scales + s.R * 64;
    w.bars = w.descs + kWideSegs * 32;
    w.misc = w.bars + (2 * s.R + 2 * kWideSegs + 2 * s.HG) * 8;
    w.total = w.misc + ((int(sizeof(WideMisc)) + 15) & ~15);
    return w;
}

struct WideDesc {  // one segment, from the producer to the consumers
    int32_t b, hg;   // sequence, head group
    int32_t j0, npg; // first listed page and pages; npg = 0 marks the end of the share
    int32_t L;
    int32_t k0, k1;  // CTAs that hold pages of (b, hg)
    int32_t pad;
};

struct WideParams {
    DecodeParams d;  // k_scale and v_scale: [NB][Hkv] for 8-bit caches
    WideShape shape;
    int32_t window, sinks;
};

__device__ __forceinline__ void cp_async4(void* smem_dst, const void* gmem_src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem_dst)), "l"(gmem_src) : "memory");
}
// Arrives on `bar` once when all of this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <class MathT, int D, int G, bool I8>
__global__ void __launch_bounds__(kWideThreads, 1) decode_wide_kernel(const __grid_constant__ WideParams wp) {
    constexpr int NT = kWideThreads, S = kWideSegs;
    constexpr int kTile = 16 * D * (I8 ? 1 : 2);
    const DecodeParams& p = wp.d;
    const WideShape& sh = wp.shape;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const WideLayout lay = wide_layout(sh, D);
    uint8_t* ring = smem + lay.ring;
    float* scales = reinterpret_cast<float*>(smem + lay.scales);  // per stage: 8 K scales, 8 V scales
    WideDesc* descs = reinterpret_cast<WideDesc*>(smem + lay.descs);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars);
    uint64_t* empty = full + sh.R;
    uint64_t* segfull = empty + sh.R;
    uint64_t* segempty = segfull + S;
    uint64_t* partfull = segempty + S;   // per head: the other parts' states are written
    uint64_t* partempty = partfull + sh.HG;  // and read
    WideMisc* misc = reinterpret_cast<WideMisc*>(smem + lay.misc);
    volatile int* abort = &misc->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int HG = sh.HG, HS = sh.HS, SPL = 1 << sh.SPL_LOG, WPH = 1 << sh.WPH_LOG, R = sh.R;

    if (warp == kWideWarps && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.tmap_v)) : "memory");
    }
    if (warp == 0) {
        for (int r = lane; r < R; r += 32) {
            mbar_init(&full[r], I8 ? 2 : 1);  // the TMA copies' expectation, and the scales' arrival
            mbar_init(&empty[r], uint32_t(HS));
        }
        if (lane < S) {
            mbar_init(&segfull[lane], 1);
            mbar_init(&segempty[lane], uint32_t(HG * WPH));
        }
        if (lane < HG) {
            mbar_init(&partfull[lane], uint32_t(WPH - 1));
            mbar_init(&partempty[lane], 1);
        }
        if (lane == 0) misc->abort = 0;
        fence_mbar_init();
    }
    // everything below reads what kernels before this one may have written
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the CTA's share: a scan of NG * (pages + seg_weight) over the sequences ----
    const bool one_chunk = p.B <= NT;
    long long v_mine = 0, incl_mine = 0, Wt = 0;
    int32_t L_mine = 0;
    auto units = [&](int32_t L) -> long long {
        return L > 0 ? (long long)(WindowPages(L, wp.window, wp.sinks).np + p.seg_weight) * p.NG : 0;
    };
    for (int base = 0; base < p.B; base += NT) {
        const int b = base + threadIdx.x;
        long long v = 0;
        if (b < p.B) {
            L_mine = clamp_len<16>(p, b, blockIdx.x == 0);
            v = units(L_mine);
            if (L_mine == 0 && (b % int(gridDim.x)) == int(blockIdx.x)) {
                uint4* o = reinterpret_cast<uint4*>(p.out + int64_t(b) * p.Hq * D);
                for (int i = 0; i < p.Hq * D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
            }
        }
        long long chunk_total;
        const long long incl = Wt + block_incl_scan<NT>(v, misc->red, chunk_total);
        Wt += chunk_total;
        v_mine = v;
        incl_mine = incl;
    }
    const int64_t want = (Wt + p.min_pages - 1) / p.min_pages;
    const int64_t grid_eff = want < int64_t(gridDim.x) ? want : int64_t(gridDim.x);
    if (Wt == 0 || int64_t(blockIdx.x) >= grid_eff) return;
    const Split split{Wt / grid_eff, Wt % grid_eff};
    const int64_t p_start = split.start(blockIdx.x), p_end = split.start(int64_t(blockIdx.x) + 1);
    auto locate = [&](int b, long long v, long long incl, int32_t L) {
        if (v > 0 && incl - v <= p_start && p_start < incl) {
            misc->b0 = b;
            misc->L0 = L;
            misc->pre0 = incl - v;
        }
    };
    if (one_chunk) {
        locate(threadIdx.x, v_mine, incl_mine, L_mine);
    } else {
        long long carry = 0;
        for (int base = 0; base < p.B; base += NT) {
            const int b = base + threadIdx.x;
            const int32_t L = b < p.B ? clamp_len<16>(p, b, false) : 0;
            const long long v = units(L);
            long long chunk_total;
            const long long incl = carry + block_incl_scan<NT>(v, misc->red, chunk_total);
            locate(b, v, incl, L);
            carry += chunk_total;
        }
    }
    __syncthreads();

    if (warp == kWideWarps) {
        // ======================= producer warp =======================
        uint32_t stage_i = 0, seg_i = 0;
        const int C = R < 32 ? R : 32;
        bool ok = true;
        const uint64_t pol = policy_evict_first();
        const uint32_t stage_tx = uint32_t(2 * HS * kTile);
        int b = misc->b0;
        int32_t L = misc->L0;
        WindowPages pages(L, wp.window, wp.sinks);
        int64_t unit = pages.np + p.seg_weight;
        int hg = int((p_start - misc->pre0) / unit);
        int64_t u0 = misc->pre0 + int64_t(hg) * unit;  // line position of (b, hg)'s first page
        while (ok && u0 < p_end) {
            const int j = cut_page(p_start, u0, pages.np, sh.snap);
            const int npg = cut_page(p_end, u0, pages.np, sh.snap) - j;
            if (npg > 0) {
                if (lane == 0) {
                    const int s = seg_i % S;
                    if (seg_i >= S) ok = mbar_wait(&segempty[s], ((seg_i / S) - 1) & 1, abort);
                    if (ok) {
                        // the CTAs of the segment's first and last page
                        int k0 = split.owner(u0), k1 = split.owner(u0 + pages.np - 1);
                        if (cut_page(split.start(k0 + 1), u0, pages.np, sh.snap) == 0) ++k0;
                        if (cut_page(split.start(k1), u0, pages.np, sh.snap) == pages.np) --k1;
                        descs[s] = WideDesc{b, hg, j, npg, L, k0, k1, 0};
                        mbar_arrive(&segfull[s]);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                // one lane per stage: HS heads' K tiles, then their V tiles
                const int32_t* bt = p.block_tables + int64_t(b) * p.M;
                const int tile0 = hg * HG;
                const int nst = npg << sh.SPL_LOG;
                for (int c0 = 0; ok && c0 < nst; c0 += C) {
                    const int n = (nst - c0) < C ? (nst - c0) : C;
                    bool lane_ok = true;
                    if (lane < n) {
                        const int x = c0 + lane;
                        int32_t blk = __ldg(bt + pages.page(j + (x >> sh.SPL_LOG)));
                        if (blk < 0 || blk >= p.NB) {
                            raise_error(PA_DEVERR_BLOCK_ID);
                            blk = 0;
                        }
                        const int sub = x & (SPL - 1);
                        const uint32_t i = stage_i + x;
                        const int slot = int(i % R);
                        const uint32_t use = i / R;
                        if (use > 0) lane_ok = mbar_wait(&empty[slot], (use - 1) & 1, abort);
                        if (lane_ok) {
                            uint8_t* st = ring + slot * 2 * sh.stage_k;
                            mbar_arrive_expect_tx(&full[slot], stage_tx);
                            const int tile = blk * p.Hkv + tile0 + sub * HS;
                            tma_load_4d(st, &p.tmap_k, 0, 0, 0, tile, &full[slot], pol);
                            tma_load_4d(st + sh.stage_k, &p.tmap_v, 0, 0, 0, tile, &full[slot], pol);
                            if constexpr (I8) {
                                float* sc = scales + slot * 16;
                                for (int h = 0; h < HS; ++h) {
                                    cp_async4(sc + h, p.k_scale + tile + h);
                                    cp_async4(sc + 8 + h, p.v_scale + tile + h);
                                }
                                cp_async_arrive(&full[slot]);
                            }
                        }
                    }
                    ok = __all_sync(0xffffffffu, lane_ok);
                }
                stage_i += nst;
                ++seg_i;
            }
            u0 += unit;
            if (u0 < p_end && ++hg == p.NG) {
                hg = 0;
                do {
                    ++b;
                    L = clamp_len<16>(p, b, false);
                } while (L == 0);
                pages = WindowPages(L, wp.window, wp.sinks);
                unit = pages.np + p.seg_weight;
            }
        }
        if (ok && lane == 0) {  // end-of-share marker
            const int s = seg_i % S;
            if (seg_i >= S) ok = mbar_wait(&segempty[s], ((seg_i / S) - 1) & 1, abort);
            if (ok) {
                descs[s].npg = 0;
                mbar_arrive(&segfull[s]);
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok && lane == 0) {
            // error path: let every copy that may have started land before
            // the CTA's shared memory is freed
            const uint32_t last = stage_i + C;
            for (uint32_t i = (last > uint32_t(R) ? last - R : 0); i < last; ++i)
                mbar_wait(&full[i % R], (i / R) & 1, nullptr, 20000000ull);
        }
        return;
    }
    if (warp >= HG << sh.WPH_LOG) return;

    // ========================= consumer warps =========================
    const int head = warp % HG, part = warp / HG;
    const int sub = head / HS, pos = head - sub * HS;  // stage of a page, tile of the stage
    uint32_t page_base = 0, seg_i = 0;
    const int64_t hgG = int64_t(HG) * G;
    float4* mine = reinterpret_cast<float4*>(smem + lay.parts + ((part - 1) * HG + head) * part_bytes(D));  // part > 0
    MathT st;

    while (true) {
        const int s = seg_i % S;
        if (!mbar_wait(&segfull[s], (seg_i / S) & 1, abort)) return;
        const WideDesc d = descs[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(&segempty[s]);
        if (d.npg == 0) break;
        const int g = d.hg * HG + head;
        const int64_t row = int64_t(d.b) * p.Hq + int64_t(g) * G;  // its first query head
        st.load_q_global(p.q + row * (D * 2), lane, p.qscale);
        st.reset();
        const WindowPages pages(d.L, wp.window, wp.sinks);
        // this part's pages: those whose running number is `part` modulo WPH,
        // so (R being a multiple of SPL * WPH) its stages recur in the same
        // slots and every parity wait is exact
        for (int k = int((part - page_base) & uint32_t(WPH - 1)); k < d.npg; k += WPH) {
            const uint32_t i = ((page_base + uint32_t(k)) << sh.SPL_LOG) + sub;
            const int slot = int(i % R);
            const int pg = pages.page(d.j0 + k);
            const uint32_t vis = visible_tokens(pg, d.L, pages.first, wp.sinks);
            if (!mbar_wait(&full[slot], (i / R) & 1, abort)) return;
            uint8_t* kt = ring + slot * 2 * sh.stage_k + pos * kTile;
            uint8_t* vt = kt + sh.stage_k;
            if constexpr (I8) {
                st.page(kt, vt, vis, scales[slot * 16 + pos], scales[slot * 16 + 8 + pos], lane);
            } else {
                if (vis != 0xffffu) {
                    // rows that do not count may hold anything (NaN included): clear them
                    // in the V tile so that 0 * row stays 0 in the tensor core
                    for (int x = lane; x < D / 64 * 128; x += 32) {
                        const int t = (x >> 3) & 15;
                        if (!((vis >> t) & 1))
                            *reinterpret_cast<uint4*>(vt + (x >> 7) * 2048 + t * 128 + (x & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                    fence_proxy_async_smem();  // before the stage is refilled by TMA
                }
                st.template page<true>(kt, vt, int(vis), lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
        }

        // ---- the parts meet: part 0 takes the others' states over in order ----
        const int first_part = int(page_base & uint32_t(WPH - 1));  // of the segment's page 0
        page_base += uint32_t(d.npg);
        auto has_pages = [&](int w) { return int((w - first_part) & (WPH - 1)) < d.npg; };
        if (part > 0) {
            if (seg_i > 0 && !mbar_wait(&partempty[head], (seg_i - 1) & 1, abort)) return;
            if (has_pages(part)) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    mine[i * 32 + lane] = make_float4(st.acc[i][0], st.acc[i][1], st.acc[i][2], st.acc[i][3]);
                mine[D / 16 * 32 + lane] = make_float4(st.m[0], st.m[1], st.l[0], st.l[1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&partfull[head]);
            ++seg_i;
            continue;
        }
        if (!mbar_wait(&partfull[head], seg_i & 1, abort)) return;
        for (int w = 1; w < WPH; ++w) {
            if (!has_pages(w)) continue;
            const float4* o =
                reinterpret_cast<const float4*>(smem + lay.parts + ((w - 1) * HG + head) * part_bytes(D));
            const float4 ml = o[D / 16 * 32 + lane];
            const float n0 = fmaxf(st.m[0], ml.x), n1 = fmaxf(st.m[1], ml.y);
            // a state that has seen no token has m = -inf and sums of 0
            const float a0 = exp2f(st.m[0] - n0), a1 = exp2f(st.m[1] - n1);
            const float w0 = exp2f(ml.x - n0), w1 = exp2f(ml.y - n1);
            st.m[0] = n0;
            st.m[1] = n1;
            st.l[0] = st.l[0] * a0 + ml.z * w0;
            st.l[1] = st.l[1] * a1 + ml.w * w1;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const float4 v = o[i * 32 + lane];
                st.acc[i][0] = st.acc[i][0] * a0 + v.x * w0;
                st.acc[i][1] = st.acc[i][1] * a1 + v.y * w1;
                st.acc[i][2] = st.acc[i][2] * a0 + v.z * w0;
                st.acc[i][3] = st.acc[i][3] * a1 + v.w * w1;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&partempty[head]);

        // ---- segment end: this (b, g)'s result, or its piece and the merge of the pieces ----
        const int nk = d.k1 - d.k0 + 1;
        const int leaf = int(blockIdx.x) - d.k0;
        int32_t* top = p.counters + int64_t(d.b) * p.Hkv + g;
        if (nk == 1) {
            st.finish();
            st.store_out(p.out + row * D, lane);
        } else if (nk <= kFastMergePieces) {
            // ticket first; the second piece to finish merges the first one's
            // published partial with its own registers, in leaf order
            if (ticket(top, nk, lane)) {
                const int64_t sl = leaf_slot(d.k0, 1 - leaf);
                const int* flag = p.slot_sync + sl * HG + head;
                const uint64_t t0 = globaltimer_ns();
                for (uint32_t it = 0; ld_acquire_gpu(flag) == 0; ++it) {  // set right after its ticket
                    __nanosleep(32);
                    if ((it & 63u) == 63u && globaltimer_ns() - t0 > kWaitLimitNs) {
                        raise_error(PA_DEVERR_TIMEOUT);
                        break;
                    }
                }
                __syncwarp();
                const int64_t ps = sl * hgG + int64_t(head) * G;
                typename MathT::Piece other;
                st.piece_load(other, p.part_o + ps * D, p.part_ml + ps, lane);
                st.finish();
                st.store_merged2(other, leaf == 0, p.out + row * D, lane);
                __syncwarp();
                if (lane == 0) {
                    p.slot_sync[sl * HG + head] = 0;
                    *top = 0;
                }
            } else {
                const int64_t ps = leaf_slot(d.k0, leaf) * hgG + int64_t(head) * G;
                st.finish();
                st.store_partial(p.part_o + ps * D, p.part_ml + ps, nullptr, nullptr, lane);
                __threadfence();
                __syncwarp();
                if (lane == 0) st_release_gpu(p.slot_sync + leaf_slot(d.k0, leaf) * HG + head, 1);
            }
        } else {
            const int64_t ps = leaf_slot(d.k0, leaf) * hgG + int64_t(head) * G;
            st.finish();
            st.store_partial(p.part_o + ps * D, p.part_ml + ps, nullptr, nullptr, lane);
            __threadfence();
            __syncwarp();
            if (nk <= kMergeFanIn) {
                if (ticket(top, nk, lane)) {
                    merge_pieces<D, G>(p, d.k0, 0, 1, nk, HG, head, lane, p.out + row * D);
                    if (lane == 0) *top = 0;
                }
            } else {
                const int first = leaf - leaf % kMergeFanIn;
                const int runs = (nk + kMergeFanIn - 1) / kMergeFanIn;
                const int in_run = nk - first < kMergeFanIn ? nk - first : kMergeFanIn;
                int32_t* gc = p.slot_sync + leaf_slot(d.k0, first) * HG + head;
                if (ticket(gc, in_run, lane)) {
                    merge_pieces<D, G>(p, d.k0, first, 1, in_run, HG, head, lane, nullptr);
                    if (lane == 0) *gc = 0;
                    __threadfence();
                    __syncwarp();
                    if (ticket(top, runs, lane)) {
                        merge_pieces<D, G>(p, d.k0, 0, kMergeFanIn, runs, HG, head, lane, p.out + row * D);
                        if (lane == 0) *top = 0;
                    }
                }
            }
        }
        ++seg_i;
    }
}

}  // namespace pa
